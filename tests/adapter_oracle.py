"""The 4-bit weight, the 8-bit checkpoint and the backward pass in 64 bits, from
their definitions in include/lynx.h, and the error bounds the tests use.

Plain torch on float64 tensors (any device); nothing here calls the library.

Rounding units: one bf16 rounding is off by at most 2^-8 of the value; a sum of
n terms in fp32 by at most n 2^-23 of the sum of magnitudes (2^-24 a rounded
addition, 2^-23 where the tensor core truncates).
"""
import torch

BF = 2.0 ** -8
F32 = 2.0 ** -23
TINY = 2.0 ** -126  # below the normal range an absolute bound


# ---- weights in 4 bits ------------------------------------------------------


def w4_quantize(W, group, zero_points):
    """(q [N,K], s [N,K/group], z [N,K/group]) in float64."""
    N, K = W.shape
    w = W.double().reshape(N, K // group, group)
    if zero_points:
        hi, lo = w.amax(2).clamp(min=0), w.amin(2).clamp(max=0)
        s = ((hi - lo) / 15).float().bfloat16().double()
        one = torch.where(s == 0, 1.0, s)
        z = torch.where(s == 0, 0.0, torch.round(-lo / one).clamp(0, 15))
    else:
        s = (w.abs().amax(2) / 7).float().bfloat16().double()
        one = torch.where(s == 0, 1.0, s)
        z = torch.full_like(s, 8.0)
    q = (torch.round(w / one[..., None]) + z[..., None]).clamp(0, 15)
    q = torch.where((s == 0)[..., None], z[..., None].expand_as(q), q)
    return q.reshape(N, K), s, z


def w4_pack(q):
    """q [N,K] in 0..15 -> bytes [N,K/2]: nibbles k = 0, 2, 4, 6, 1, 3, 5, 7 of each word."""
    n = q.to(torch.int64).reshape(q.shape[0], -1, 8)[..., [0, 2, 4, 6, 1, 3, 5, 7]]
    return (n[..., 0::2] + 16 * n[..., 1::2]).reshape(q.shape[0], -1).to(torch.uint8)


def w4_values(q, s, z):
    N, K = q.shape
    per = K // s.shape[1]
    return (q - z.repeat_interleave(per, 1)) * s.repeat_interleave(per, 1)


def gelu(v):
    return v * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (v + 0.044715 * v ** 3))


def linear_w4(X, W, bias=None, A=None, B=None, act=False):
    """(Y, bound on |error|) for W [N,K] float64 values."""
    X = X.double()
    K = X.shape[1]
    y, size, n = X @ W.t(), X.abs() @ W.abs().t(), K + 16
    if A is not None:
        A, B = A.double(), B.double()
        y = y + (X @ A.t()) @ B.t()
        size = size + (X.abs() @ A.abs().t()) @ B.abs().t()
        n += A.shape[0]
    if bias is not None:
        y = y + bias.double()
        size = size + bias.double().abs()
    tol = n * F32 * size
    if act:  # slope at most 1.13; the hardware exponential and reciprocal: a few fp32 units
        y = gelu(y)
        tol = 1.13 * tol + 2.0 ** -18 * y.abs()
    return y, tol + BF * y.abs() + TINY


# ---- checkpoints ------------------------------------------------------------


def log2_floor(v):
    """floor(log2 v) of positive float64 (frexp is exact; a device's log2 need not be at powers of two)."""
    return (torch.frexp(v)[1] - 1).double()


def ckpt8_store(X, int8):
    """(q [M,K] float64 values of the stored numbers, e [M,K/32] int64 bytes)."""
    x = X.double()
    M, K = x.shape
    b = x.reshape(M, -1, 32)
    top = b.abs().amax(2)
    bad = ~torch.isfinite(top)
    top = torch.where(bad, 0.0, top)
    lead = log2_floor(top.clamp(min=2.0 ** -140))
    if int8:
        e = lead.clamp(min=-127)
        q = torch.round(b / torch.exp2(e - 6)[..., None]).clamp(-127, 127)
    else:
        e = (lead - 8 + (top > 448 * torch.exp2(lead - 8))).clamp(min=-127)
        v = b / torch.exp2(e)[..., None]
        step = torch.exp2(log2_floor(v.abs().clamp(min=2.0 ** -6)) - 3)
        most = torch.where(e == 120, 240.0, 448.0)[..., None]
        q = torch.minimum(torch.maximum(torch.round(v / step) * step, -most), most)
    q = torch.where(bad[..., None], 0.0, q)
    e = torch.where(bad, 255, (e + 127).long())
    return q.reshape(M, K), e


def ckpt8_values(q, e, int8):
    per = torch.exp2(e.double() - (133 if int8 else 127))
    per = torch.where(e == 255, torch.nan, per)
    return q.double() * per.repeat_interleave(32, 1)


# ---- backward ---------------------------------------------------------------


def lora_backward(dY, x, A, B):
    """{name: (value, bound on |error|)}; T and dT are rounded to bf16 before their second product."""
    dY, A, B = dY.double(), A.double(), B.double()
    M, N = dY.shape
    K = x.shape[1]
    T, dT = x @ A.t(), dY @ B
    dT_sum = (N + 16) * F32 * (dY.abs() @ B.abs())
    T_off = BF * T.abs() + (K + 16) * F32 * (x.abs() @ A.abs().t())
    dT_off = BF * dT.abs() + dT_sum
    dB, dA = dY.t() @ T, dT.t() @ x
    dB_tol = BF * dB.abs() + dY.abs().t() @ T_off + (M + 16) * F32 * (dY.abs().t() @ (T.abs() + T_off))
    dA_tol = BF * dA.abs() + dT_off.t() @ x.abs() + (M + 16) * F32 * ((dT.abs() + dT_off).t() @ x.abs())
    # twice the last rounding where a sum's own error crosses a binade
    return {"dA": (dA, 1.01 * dA_tol + TINY), "dB": (dB, 1.01 * dB_tol + TINY), "dT": (dT, 1.01 * dT_off + TINY)}


def keep(x):
    """The 2:4 selection of x [M,K] (0 or 1): two largest magnitudes of 4, ties to the lower position."""
    M, K = x.shape
    a = x.abs().reshape(M, -1, 4)
    first = torch.argsort(a, dim=2, descending=True, stable=True)[..., :2]
    return torch.zeros_like(a).scatter_(2, first, 1.0).reshape(M, K)


def sparsify(x):
    m = keep(x)
    L, Lk = x.abs().sum(1, keepdim=True), (m * x.abs()).sum(1, keepdim=True)
    s = torch.where(Lk > 0, L / torch.where(Lk > 0, Lk, 1.0), 1.0)
    return s * m * x


def sparsify_backward(G, x, dT=None, A=None):
    """(dX, bound on |error|)."""
    G = G.double()
    K = x.shape[1]
    m = keep(x)
    L, Lk = x.abs().sum(1, keepdim=True), (m * x.abs()).sum(1, keepdim=True)
    some = Lk > 0
    safe = torch.where(some, Lk, 1.0)
    s = torch.where(some, L / safe, 1.0)
    D = (m * G * x).sum(1, keepdim=True)
    second = torch.where(some, torch.sign(x) * (D / safe) * (1 - s * m), 0.0)
    dX = s * m * G + second
    size = s * m * G.abs() + (m * (G * x).abs()).sum(1, keepdim=True) / safe * (1 + s * m)
    tol = 2 * (K + 16) * F32 * size
    if dT is not None:
        dT, A = dT.double(), A.double()
        dX = dX + dT @ A
        tol = tol + (A.shape[0] + 16) * F32 * (dT.abs() @ A.abs())
    return dX, 1.01 * (BF * dX.abs() + tol) + TINY
