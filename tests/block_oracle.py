"""Layer norm, the residual epilogue and their backward passes in 64 bits, written
from the formulas in include/lynx.h, with the error that fp32 arithmetic and one
bf16 rounding may leave.

BF16 is half a step of bf16 relative to the value.  SUM bounds the fp32 rounding of
one sum relative to the sum of its terms' magnitudes: each addition is off by at
most 2^-24, and no chain of additions in these kernels is longer than 128.
"""
import math

import torch

BF16 = torch.finfo(torch.bfloat16).eps / 2
SUM = 128 * 2.0 ** -24


def layer_norm(X, weight, bias, eps):
    """{name: (value, tolerance)} of Y, mean and rstd."""
    x = X.double()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = ((d * d).mean(1) + eps) ** -0.5
    xh = d * rstd[:, None]
    w = torch.ones(X.shape[1], dtype=torch.float64, device=X.device) if weight is None else weight.double()
    b = torch.zeros_like(w) if bias is None else bias.double()
    y = xh * w + b
    mean_tol = SUM * x.abs().mean(1)
    # the variance: its own sum, and the square of the mean's error; rsqrt is off by 2 ulp at most
    rstd_rel = SUM + 0.5 * (mean_tol * rstd) ** 2 + 2.0 ** -22
    y_tol = BF16 * y.abs() + (mean_tol * rstd)[:, None] * w.abs() + (xh * w).abs() * (rstd_rel + SUM)[:, None] + SUM * b.abs()
    return {"Y": (y, y_tol), "mean": (mean, mean_tol), "rstd": (rstd, rstd * rstd_rel)}


def layer_norm_backward(dY, X, mean, rstd, weight, dR):
    dy, x = dY.double(), X.double()
    K = x.shape[1]
    w = torch.ones(K, dtype=torch.float64, device=X.device) if weight is None else weight.double()
    r = rstd.double()[:, None]
    xh = (x - mean.double()[:, None]) * r
    g = dy * w
    a, c = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - a - xh * c)
    # xh itself: the difference and the product, 2^-23 of it; the rest: the two sums and a few products
    size = r * (g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    if dR is not None:
        dx = dx + dR.double()
    return {"dX": (dx, BF16 * dx.abs() + 2 * SUM * size),
            "dweight": column_sum(dy * xh), "dbias": column_sum(dy)}


def column_sum(terms, terms_tol=None):
    s = terms.sum(0)
    tol = BF16 * s.abs() + 2 * SUM * terms.abs().sum(0)
    return s, tol if terms_tol is None else tol + terms_tol.sum(0)


def gelu(z):
    return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))


def gelu_slope(z):
    c = 2 * math.sqrt(2 / math.pi)
    s = torch.sigmoid(c * (z + 0.044715 * z ** 3))
    return s + z * s * (1 - s) * c * (1 + 3 * 0.044715 * z ** 2)


def act_backward(dY, Z):
    """The slope is off by 2^-19 at most: the exponent's argument u by 2^-22 |u|, which
    sig (1 - sig) |u| (1 + |z| a') < 1 turns into 2^-22 of the slope's terms, the base-2
    exponential, the reciprocal and five roundings of values below 2 by 2^-21."""
    dy = dY.double()
    dz = dy * gelu_slope(Z.double())
    off = 2.0 ** -19 * dy.abs()
    return {"dZ": (dz, BF16 * dz.abs() + off), "dbias": column_sum(dz, off)}


def selected(X):
    """S(X): of each 4 the two of largest magnitude (ties to the lower position), times sum|x| / sum|kept|."""
    x = X.double()
    M, K = x.shape
    top = torch.sort(x.abs().reshape(M, -1, 4), dim=2, descending=True, stable=True).indices[..., :2]
    m = torch.zeros(M, K // 4, 4, dtype=torch.float64, device=X.device).scatter_(2, top, 1.0).reshape(M, K)
    held = (m * x.abs()).sum(1)
    s = torch.where(held > 0, x.abs().sum(1) / held, torch.ones_like(held))
    return m * x * s[:, None]


def linear_residual(X, W, bias, A, B, R, skip, act):
    """W may be [N,K] of any type (a weight in 4 bits as the values it stands for)."""
    x, w = X.double(), W.double()
    K = x.shape[1]
    sx = x if skip else selected(X)
    p = sx @ w.t()
    # the tensor cores add 16 products at a time, each addition off by 2^-23 at most of what is there
    tol = (K / 16 + 64) * 2.0 ** -23 * (sx.abs() @ w.abs().t())
    if A is not None:
        t = x @ A.double().t()
        p = p + t @ B.double().t()
        # T is rounded to bf16 on its way into the second product
        tol = tol + 1.01 * BF16 * (t.abs() @ B.double().abs().t()) + \
            (K / 16 + 64) * 2.0 ** -23 * ((x.abs() @ A.double().abs().t()) @ B.double().abs().t())
    if bias is not None:
        p = p + bias.double()
        tol = tol + 2.0 ** -23 * bias.double().abs()
    y, y_tol = p, tol
    if act:  # |gelu'| < 1.13
        y, y_tol = gelu(p), 1.13 * tol + 2.0 ** -20 * p.abs()
    if R is not None:
        y = y + R.double()
    return {"Y": (y, BF16 * (y.abs() + y_tol) + y_tol), "Z": (p, BF16 * (p.abs() + tol) + tol)}


def check(got, want, what=""):
    value, tol = want
    assert got.shape == value.shape, what
    off = (got.double() - value).abs()
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / tol.clamp_min(1e-300)).max()):.3g} " \
                          f"times the tolerance at {bad.nonzero()[0].tolist()}"
