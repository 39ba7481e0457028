"""What is measured of the layer's 4-bit, checkpoint and backward operators.

Five operators around the layer Y = act(S(X) W^T + bias + (X A^T) B^T):

* linear_w4          a few tokens through a frozen weight kept in 4 bits with
                     group scales, LoRA branch, bias and activation included
* w4_weights         a weight taken to 4 bits and back (what a user does once
                     per layer, and again where prompts go through lynx_linear)
* ckpt8              an activation taken to 8 bits with a power-of-two scale per
                     32 values, and back (what is kept of X for the backward pass)
* lora_backward      dT = dY B, dB = dY^T T, dA = dT^T X with T = X A^T and X
                     the 8-bit checkpoint
* sparsify_backward  the gradient through the 2:4 selection and its row
                     compensation at the checkpoint, plus the branch's dT A

``own`` false: plain torch in 32 bits (64 next to borders), rounded once at the
end.  ``own`` true: the calls a user makes of the framework.
"""
import math

import torch

own = False

DEV = "cuda"
BF = torch.bfloat16


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # one token through a small projection (a time-embedding layer): latency
        {"name": "w4_one_token_small", "op": "linear_w4", "M": 1, "N": 512, "K": 512, "group": 64, "zeros": False,
         "r": 0, "bias": True, "act": False},
        # one token through the MLP up-projection, adapter and GELU included
        {"name": "w4_one_token_up", "op": "linear_w4", "M": 1, "N": 12288, "K": 4096, "group": 128, "zeros": True,
         "r": 64, "bias": True, "act": True},
        # five sequences' tokens through the down-projection, fine groups
        {"name": "w4_five_tokens_down", "op": "linear_w4", "M": 5, "N": 4104, "K": 12288, "group": 32, "zeros": False,
         "r": 64, "bias": True, "act": False},
        # a decoding batch of 32 through QKV
        {"name": "w4_batch_qkv", "op": "linear_w4", "M": 32, "N": 9216, "K": 4096, "group": 128, "zeros": False,
         "r": 64, "bias": True, "act": False},
        # the weight of an odd-sized layer, and of a full one
        {"name": "w4_weights_odd", "op": "w4_weights", "N": 1000, "K": 576, "group": 64, "zeros": False},
        {"name": "w4_weights_up", "op": "w4_weights", "N": 12288, "K": 4096, "group": 128, "zeros": True},
        # the checkpoint of a short ragged batch, and of the down-projection's input
        {"name": "ckpt8_ragged", "op": "ckpt8", "M": 300, "K": 576, "format": "int8", "kind": "mixture"},
        {"name": "ckpt8_down", "op": "ckpt8", "M": 4608, "K": 12288, "format": "e4m3", "kind": "gelu"},
        # adapter gradients of a short ragged batch, and of the MLP up-projection
        {"name": "lora_backward_ragged", "op": "lora_backward", "M": 300, "N": 1000, "K": 576, "r": 16,
         "format": "e4m3"},
        {"name": "lora_backward_up", "op": "lora_backward", "M": 4608, "N": 12288, "K": 4096, "r": 64,
         "format": "int8"},
        # the input gradient of a short ragged batch without an adapter, and of the down-projection
        {"name": "sparsify_backward_ragged", "op": "sparsify_backward", "M": 257, "K": 1088, "r": 0,
         "format": "e4m3", "kind": "mixture"},
        {"name": "sparsify_backward_down", "op": "sparsify_backward", "M": 4608, "K": 12288, "r": 64,
         "format": "int8", "kind": "gelu"},
    ]


def _log(rng, lo, hi, step):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(max(round(v / step) * step, lo), hi))


def draw(rng):
    op = rng.choice(["linear_w4", "linear_w4", "w4_weights", "ckpt8", "lora_backward", "lora_backward",
                     "sparsify_backward", "sparsify_backward"])
    fmt = rng.choice(["int8", "e4m3"])
    kind = rng.choice(["mixture", "gelu"])
    if op == "linear_w4":
        g = rng.choice([32, 64, 128])
        return {"op": op, "M": rng.randint(1, 32), "N": _log(rng, 512, 9216, 8), "K": _log(rng, 512, 4096, max(g, 64)),
                "group": g, "zeros": rng.random() < 0.5, "r": rng.choice([0, 16, 64, 64, 144, 256]),
                "bias": rng.random() < 0.7, "act": rng.random() < 0.3}
    if op == "w4_weights":
        g = rng.choice([32, 64, 128])
        return {"op": op, "N": _log(rng, 512, 12288, 8), "K": _log(rng, 512, 4096, max(g, 64)), "group": g,
                "zeros": rng.random() < 0.5}
    if op == "ckpt8":
        return {"op": op, "M": _log(rng, 128, 4608, 1), "K": _log(rng, 512, 12288, 64), "format": fmt, "kind": kind}
    if op == "lora_backward":
        r = rng.choice([16, 32, 64, 64, 112, 256])
        return {"op": op, "M": _log(rng, 128, 4608 if r <= 64 else 1024, 1), "N": _log(rng, 512, 9216, 8),
                "K": _log(rng, 512, 4096, 64), "r": r, "format": fmt}
    return {"op": op, "M": _log(rng, 128, 4608, 1), "K": _log(rng, 512, 12288, 64), "r": rng.choice([0, 16, 32, 64]),
            "format": fmt, "kind": kind}


# ---------------------------------------------------------------------------
# inputs: the distributions of the layer's own workloads


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std


def _activations(g, M, K, kind):
    """A heavy-tailed mixture (8 % N(0, 1), the rest N(0, 0.05)), or GELU of N(-0.5, 1)."""
    z = _normal(g, (M, K), 1.0)
    if kind == "gelu":
        z = z - 0.5
        z = 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    else:
        large = torch.rand((M, K), generator=g, device=DEV) < 0.08
        z = torch.where(large, z, z * 0.05)
    return z.to(BF)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case, "op": case["op"]}
    op = case["op"]
    if op in ("linear_w4", "w4_weights"):
        N, K = case["N"], case["K"]
        W = _normal(g, (N, K), 1.0 / math.sqrt(K)).to(BF)
        if op == "w4_weights":
            s["W"] = W
            return s
        M, r = case["M"], case["r"]
        q, s["scales"], s["zeros"] = _w4_split(W, case["group"], case["zeros"])
        s["Wq"] = _w4_pack(q)
        s["X"] = _activations(g, M, K, "mixture")
        s["bias"] = _normal(g, (N,), 0.02).to(BF) if case["bias"] else None
        s["A"] = _normal(g, (r, K), 0.01).to(BF) if r else None
        s["B"] = _normal(g, (N, r), 0.01).to(BF) if r else None
        return s
    M, K = case["M"], case["K"]
    X = _activations(g, M, K, case.get("kind", "mixture"))
    if op == "ckpt8":
        s["X"] = X
        return s
    r = case["r"]
    s["q"], s["e"] = _ckpt8_split(X, case["format"])
    if op == "lora_backward":
        N = case["N"]
        s["dY"] = _normal(g, (M, N), 1e-3).to(BF)
        s["A"] = _normal(g, (r, K), 0.01).to(BF)
        s["B"] = _normal(g, (N, r), 0.01).to(BF)
        return s
    s["G"] = _normal(g, (M, K), 1e-3).to(BF)
    s["dT"] = _normal(g, (M, r), 1e-3).to(BF) if r else None
    s["A"] = _normal(g, (r, K), 0.01).to(BF) if r else None
    return s


# ---------------------------------------------------------------------------
# plain forms


def _w4_split(W, group, zeros):
    """Unsigned 4-bit values [N,K], scales [K/group, N] bf16, zero points [K/group, N] u8 or None.

    Symmetric: s = bf16(max|w| / 7), q = clamp(rint(w / s), -8, 7) + 8 (zero point 8).
    With zero points: s = bf16((hi - lo) / 15) over the group and zero, z = rint(-lo / s),
    q = clamp(rint(w / s) + z, 0, 15).  In 64 bits: rint sits next to borders."""
    N, K = W.shape
    w = W.double().view(N, K // group, group)
    if zeros:
        hi = w.amax(-1).clamp_min(0.0)
        lo = w.amin(-1).clamp_max(0.0)
        sc = ((hi - lo) / 15.0).to(torch.float32).to(BF)
        safe = torch.where(sc == 0, torch.ones_like(sc), sc).double()
        z = torch.round(-lo / safe).clamp(0, 15)
        z = torch.where(sc == 0, torch.zeros_like(z), z)
        q = (torch.round(w / safe[..., None]) + z[..., None]).clamp(0, 15)
        q = torch.where((sc == 0)[..., None], torch.zeros_like(q), q)
        return q.to(torch.uint8).view(N, K), sc.t().contiguous(), z.to(torch.uint8).t().contiguous()
    sc = (w.abs().amax(-1) / 7.0).to(torch.float32).to(BF)
    safe = torch.where(sc == 0, torch.ones_like(sc), sc).double()
    q = torch.round(w / safe[..., None]).clamp(-8, 7) + 8
    q = torch.where((sc == 0)[..., None], torch.full_like(q, 8), q)
    return q.to(torch.uint8).view(N, K), sc.t().contiguous(), None


# the place of each nibble of a 32-bit word of 8 consecutive values: low to
# high they hold k = 0, 2, 4, 6, 1, 3, 5, 7
_NIBBLES = [0, 2, 4, 6, 1, 3, 5, 7]


def _w4_pack(q):
    N, K = q.shape
    n = q.view(N, K // 8, 8)[:, :, _NIBBLES].reshape(N, K // 2, 2)
    return (n[..., 0] | (n[..., 1] << 4)).contiguous()


def _w4_unpack(Wq):
    N, K2 = Wq.shape
    n = torch.stack([Wq & 15, Wq >> 4], dim=-1).view(N, K2 // 4, 8)
    back = [_NIBBLES.index(k) for k in range(8)]
    return n[:, :, back].reshape(N, 2 * K2)


def _w4_values(q, scales, zeros):
    """(q - z) * s in 32 bits (exact: at most 5 times 8 significant bits)."""
    N, K = q.shape
    kg = scales.shape[0]
    v = q.view(N, kg, K // kg).float()
    z = zeros.t().float()[..., None] if zeros is not None else 8.0
    return ((v - z) * scales.t().float()[..., None]).view(N, K)


def _block_exponent(X, fmt):
    """Per 32 values: the power of two of the block, and which blocks hold a value that is not finite."""
    M, K = X.shape
    x = X.float().view(M, K // 32, 32)
    top = x.abs().amax(-1)
    bad = ~torch.isfinite(top)
    m, ex = torch.frexp(torch.where(bad, torch.zeros_like(top), top).double())
    ex = ex - 1  # top = (2 m) 2^ex, 1 <= 2 m < 2
    if fmt == "int8":
        e = ex  # values are multiples of 2^(e - 6)
    else:
        e = torch.where(m > 0.875, ex - 7, ex - 8)  # smallest e with top <= 448 * 2^e
    e = torch.where(top == 0, torch.full_like(e, -127), e)
    return x, e.clamp(-127, 127), bad


def _ckpt8_split(X, fmt):
    """8-bit values [M,K] (int8 or e4m3) and biased exponents [M,K/32] u8 (255: the block was not finite)."""
    M, K = X.shape
    x, e, bad = _block_exponent(X, fmt)
    x = torch.where(bad[..., None], torch.zeros_like(x), x).double()
    if fmt == "int8":
        q = torch.round(x * torch.exp2((6 - e).double())[..., None]).clamp(-127, 127).to(torch.int8)
    else:
        most = torch.where(e == 120, 240.0, 448.0).double()[..., None]  # 256 * 2^120 is not a finite bf16
        q = (x * torch.exp2(-e.double())[..., None]).clamp(-most, most).to(torch.float32).to(torch.float8_e4m3fn)
    e = torch.where(bad, torch.full_like(e, 128), e) + 127
    return q.view(M, K), e.to(torch.uint8)


def _ckpt8_values(q, e):
    """The values a checkpoint stands for, in 32 bits (exact)."""
    M, K = q.shape
    shift = 133 if q.dtype == torch.int8 else 127
    x = q.view(M, K // 32, 32).double() * torch.exp2(e.double() - shift)[..., None]
    x = torch.where((e == 255)[..., None], torch.full_like(x, float("nan")), x)
    return x.to(torch.float32).view(M, K)


def _gelu(v):
    return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))


def _keep(ax):
    """Of each 4 the two of largest magnitude, ties to the lower index."""
    a = ax.view(*ax.shape[:-1], -1, 4)
    lower = torch.ones(4, 4, dtype=torch.bool, device=ax.device).tril(-1)  # [i, j]: j < i
    ahead = (a[..., None, :] > a[..., :, None]) | ((a[..., None, :] == a[..., :, None]) & lower)
    return (ahead.sum(-1) < 2).view_as(ax)


def _plain(s):
    case, op = s["case"], s["op"]
    if op == "w4_weights":
        q, scales, zeros = _w4_split(s["W"], case["group"], case["zeros"])
        Wq = _w4_pack(q)
        W = _w4_values(_w4_unpack(Wq), scales, zeros).to(BF)
        return {"W": W, "scales": scales, "zeros": zeros}
    if op == "linear_w4":
        W = _w4_values(_w4_unpack(s["Wq"]), s["scales"], s["zeros"])
        x = s["X"].float()
        y = x @ W.t()
        if s["A"] is not None:
            y = y + (x @ s["A"].float().t()) @ s["B"].float().t()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        return (_gelu(y) if case["act"] else y).to(BF)
    if op == "ckpt8":
        return _ckpt8_values(*_ckpt8_split(s["X"], case["format"])).to(BF)
    x = _ckpt8_values(s["q"], s["e"])
    if op == "lora_backward":
        dy, A, B = s["dY"].float(), s["A"].float(), s["B"].float()
        dT = dy @ B
        dB = dy.t() @ (x @ A.t())
        dA = dT.t() @ x
        return {"dA": dA.to(BF), "dB": dB.to(BF), "dT": dT.to(BF)}
    g = s["G"].float()
    ax = x.abs()
    keep = _keep(ax)
    kept = (ax * keep).sum(-1, keepdim=True)
    some = kept > 0
    safe = torch.where(some, kept, torch.ones_like(kept))
    comp = torch.where(some, ax.sum(-1, keepdim=True) / safe, torch.ones_like(kept))
    d = (g * x * keep).sum(-1, keepdim=True)
    dx = torch.where(keep, comp * g, torch.zeros_like(g))
    dx = dx + torch.sign(x) * (d / safe) * (1.0 - comp * keep)
    if s["dT"] is not None:
        dx = dx + s["dT"].float() @ s["A"].float()
    return dx.to(BF)


# ---------------------------------------------------------------------------
# the framework's calls


def _own(s):
    from activation_sparse_gemm_lynx_b200 import lynx

    case, op = s["case"], s["op"]
    if op == "w4_weights":
        Wq, scales, zeros = lynx.lynx_w4_quantize(s["W"], group=case["group"], zero_points=case["zeros"])
        return {"W": lynx.lynx_w4_dequantize(Wq, scales, zeros), "scales": scales, "zeros": zeros}
    if op == "linear_w4":
        act = lynx.LYNX_ACT_GELU_TANH if case["act"] else lynx.LYNX_ACT_NONE
        return lynx.lynx_linear_w4(s["X"], s["Wq"], s["scales"], s["zeros"], s["bias"], s["A"], s["B"], act=act)
    if op == "ckpt8":
        fmt = lynx.LYNX_CKPT8_INT8 if case["format"] == "int8" else lynx.LYNX_CKPT8_E4M3
        q, e = lynx.lynx_ckpt8_store(s["X"], format=fmt)
        return lynx.lynx_ckpt8_restore(q, e)
    if op == "lora_backward":
        dA, dB, dT = lynx.lynx_lora_backward(s["dY"], s["q"], s["e"], s["A"], s["B"])
        return {"dA": dA, "dB": dB, "dT": dT}
    return lynx.lynx_sparsify_backward(s["G"], s["q"], s["e"], s["dT"], s["A"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# work


def work(case):
    op = case["op"]
    if op in ("linear_w4", "w4_weights"):
        N, K = case["N"], case["K"]
        side = N * (K // case["group"]) * (3 if case["zeros"] else 2)
        if op == "w4_weights":
            # quantise: read W, write the packed weight; dequantise: read that, write W
            return {"bytes": 2 * (2 * N * K + N * K // 2 + side), "flops": 4 * N * K}
        M, r = case["M"], case["r"]
        b = N * K // 2 + side + 2 * M * K + 2 * M * N + 2 * r * (N + K) + (2 * N if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * M * N * K + 2 * M * r * (N + K)}
    M, K = case["M"], case["K"]
    ckpt = M * K + M * K // 32
    if op == "ckpt8":
        return {"bytes": 2 * (2 * M * K + ckpt), "flops": 4 * M * K}
    r = case["r"]
    if op == "lora_backward":
        N = case["N"]
        return {"bytes": 2 * M * N + ckpt + 2 * 2 * r * (N + K) + 2 * M * r, "flops": 4 * M * r * (N + K)}
    return {"bytes": 2 * 2 * M * K + ckpt + 2 * r * (M + K), "flops": 10 * M * K + 2 * M * K * r}


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def _exact_w4(case, st):
    if case["op"] == "w4_weights":
        W = st["W"].double()
        N, K = W.shape
        g = W.reshape(N, -1, case["group"])
        if case["zeros"]:
            top = torch.maximum(g.max(dim=2).values, torch.zeros((), dtype=torch.float64, device=DEV))
            low = torch.minimum(g.min(dim=2).values, torch.zeros((), dtype=torch.float64, device=DEV))
            sc = ((top - low) / 15).float().bfloat16().double()
            z = torch.clamp(torch.round(-low / sc), 0, 15).nan_to_num(0.0)
            v = torch.clamp(torch.round(g / sc[:, :, None]).nan_to_num(0.0) + z[:, :, None], 0, 15) - z[:, :, None]
            zeros = z.to(torch.uint8).t().contiguous()
        else:
            sc = (g.abs().max(dim=2).values / 7).float().bfloat16().double()
            v = torch.clamp(torch.round(g / sc[:, :, None]).nan_to_num(0.0), -8, 7)
            zeros = None
        return {"W": (v * sc[:, :, None]).reshape(N, K), "scales": sc.t().contiguous(), "zeros": zeros}
    N, K = st["Wq"].shape[0], 2 * st["Wq"].shape[1]
    word = st["Wq"].reshape(N, K // 8, 4).long()
    word = word[..., 0] + (word[..., 1] << 8) + (word[..., 2] << 16) + (word[..., 3] << 24)
    place = torch.tensor([0, 4, 1, 5, 2, 6, 3, 7], device=DEV)  # the nibble of k = 0..7
    q = ((word[..., None] >> (4 * place)) & 15).reshape(N, K).double()
    per = K // st["scales"].shape[0]
    z = st["zeros"].double() if st["zeros"] is not None else torch.full_like(st["scales"], 8, dtype=torch.float64)
    W = (q - z.t().repeat_interleave(per, dim=1)) * st["scales"].double().t().repeat_interleave(per, dim=1)
    X = st["X"].double()
    Y = torch.einsum("mk,nk->mn", X, W)
    if st["A"] is not None:
        Y += torch.einsum("mr,nr->mn", torch.einsum("mk,rk->mr", X, st["A"].double()), st["B"].double())
    if st["bias"] is not None:
        Y += st["bias"].double()
    if case["act"]:
        Y = Y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (Y + 0.044715 * Y ** 3))
    return Y


def _exact_checkpoint(X, fmt):
    """X through 8 bits, by the definition, value by value in 64 bits."""
    x = X.double()
    M, K = x.shape
    big = x.reshape(M, -1, 32).abs().max(dim=2).values.repeat_interleave(32, dim=1)
    lead = torch.frexp(big.clamp_min(2.0 ** -133)).exponent.double() - 1
    if fmt == "int8":
        step = torch.exp2(lead.clamp_min(-127.0) - 6)
        return torch.clamp(torch.round(x / step), -127, 127) * step
    e = (lead - 8 + (big > 448 * torch.exp2(lead - 8))).clamp_min(-127.0)
    v = x / torch.exp2(e)
    step = torch.exp2(torch.frexp(v.abs().clamp_min(2.0 ** -6)).exponent.double() - 4)
    most = torch.where(e == 120, 240.0, 448.0).double()
    return torch.clamp(torch.round(v / step) * step, -most, most) * torch.exp2(e)


def _exact_restored(q, e):
    per = torch.exp2(e.double() - 127).repeat_interleave(32, dim=1)
    return q.double() * per / (64.0 if q.dtype == torch.int8 else 1.0)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("linear_w4", "w4_weights"):
        return _exact_w4(case, st)
    if op == "ckpt8":
        return _exact_checkpoint(st["X"], case["format"])
    X = _exact_restored(st["q"], st["e"])
    if op == "lora_backward":
        dY, A, B = st["dY"].double(), st["A"].double(), st["B"].double()
        dT = torch.einsum("mn,nr->mr", dY, B)
        T = torch.einsum("mk,rk->mr", X, A)
        return {"dA": torch.einsum("mr,mk->rk", dT, X), "dB": torch.einsum("mn,mr->nr", dY, T), "dT": dT}
    G = st["G"].double()
    M, K = X.shape
    order = torch.sort(X.abs().reshape(M, -1, 4), dim=2, descending=True, stable=True).indices[..., :2]
    m = torch.zeros(M, K // 4, 4, dtype=torch.float64, device=DEV).scatter_(2, order, 1.0).reshape(M, K)
    everything = X.abs().sum(dim=1, keepdim=True)
    held = (m * X.abs()).sum(dim=1, keepdim=True)
    s = torch.where(held > 0, everything / held, torch.ones_like(held))
    along = (G * m * X).sum(dim=1, keepdim=True)
    # d/dx of s m x: s m g, and through s = sum|x| / sum m|x|
    ds = torch.where(held > 0, torch.sign(X) / held - m * torch.sign(X) * everything / held ** 2, torch.zeros_like(X))
    dX = s * m * G + along * ds
    if st["dT"] is not None:
        dX = dX + torch.einsum("mr,rk->mk", st["dT"].double(), st["A"].double())
    return dX
