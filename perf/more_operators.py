"""What is measured of the operators before and after the layer.

Four operators of a transformer block around the layer
P = S(X) W^T + bias + (X A^T) B^T:

* layer_norm           what makes the layer's X from the residual stream
* layer_norm_backward  its input gradient, with the residual branch's gradient
                       added, and the reduction of the weight's and the bias's
* linear_residual      Y = R + act(P), with P itself kept in bf16 (Z) where a
                       backward pass follows; S(X) (path "sparse"), the dense
                       X of a skipped layer ("dense"), or a few tokens on the
                       weight in 4 bits ("w4")
* act_backward         dZ = dY act'(Z) and the bias's gradient

``own`` false: plain torch in 32 bits, rounded once at the end.  ``own`` true:
the calls a user makes of the framework.
"""
import math

import torch

own = False

DEV = "cuda"
BF = torch.bfloat16
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # one token of a decoding step before its QKV projection: latency
        {"name": "norm_one_token", "op": "layer_norm", "M": 1, "K": 4096, "affine": True, "stats": False},
        # a short ragged batch, no affine part (what a modulated block applies first), statistics kept
        {"name": "norm_ragged", "op": "layer_norm", "M": 300, "K": 1088, "affine": False, "stats": True},
        # a training batch of the MLP half
        {"name": "norm_tokens", "op": "layer_norm", "M": 4608, "K": 4096, "affine": True, "stats": True},
        # the gradients of a short ragged batch without a residual branch, and of a training batch with one
        {"name": "norm_backward_ragged", "op": "layer_norm_backward", "M": 257, "K": 576, "affine": True, "dR": False},
        {"name": "norm_backward_tokens", "op": "layer_norm_backward", "M": 4608, "K": 4096, "affine": True, "dR": True},
        # a short ragged batch through a small layer
        {"name": "residual_ragged", "op": "linear_residual", "path": "sparse", "M": 300, "N": 1000, "K": 576, "r": 16,
         "bias": True, "R": True, "Z": False, "act": False},
        # the MLP up-projection of a training step: GELU, and Z for the backward pass
        {"name": "residual_up", "op": "linear_residual", "path": "sparse", "M": 4608, "N": 12288, "K": 4096, "r": 64,
         "bias": True, "R": False, "Z": True, "act": True},
        # the MLP down-projection into the residual stream
        {"name": "residual_down", "op": "linear_residual", "path": "sparse", "M": 4608, "N": 4096, "K": 12288, "r": 64,
         "bias": True, "R": True, "Z": False, "act": False},
        # the attention output of a layer that stays dense
        {"name": "residual_out_dense", "op": "linear_residual", "path": "dense", "M": 4096, "N": 4096, "K": 4096,
         "r": 64, "bias": True, "R": True, "Z": False, "act": False},
        # one token through the down-projection, the weight in 4 bits
        {"name": "residual_one_token", "op": "linear_residual", "path": "w4", "M": 1, "N": 4096, "K": 12288, "r": 64,
         "bias": True, "R": True, "Z": False, "act": False, "group": 128},
        # the bias's gradient of a short ragged batch, and the GELU's of the MLP up-projection
        {"name": "act_backward_ragged", "op": "act_backward", "M": 300, "N": 1000, "act": True, "dbias": True},
        {"name": "act_backward_up", "op": "act_backward", "M": 4608, "N": 12288, "act": True, "dbias": True},
    ]


def _log(rng, lo, hi, step):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(max(round(v / step) * step, lo), hi))


def draw(rng):
    op = rng.choice(["layer_norm", "layer_norm_backward", "layer_norm_backward", "linear_residual", "linear_residual",
                     "linear_residual", "act_backward"])
    if op == "layer_norm":
        return {"op": op, "M": _log(rng, 1, 4608, 1), "K": _log(rng, 64, 8192, 8), "affine": rng.random() < 0.7,
                "stats": rng.random() < 0.7}
    if op == "layer_norm_backward":
        return {"op": op, "M": _log(rng, 1, 4608, 1), "K": _log(rng, 64, 8192, 8), "affine": rng.random() < 0.8,
                "dR": rng.random() < 0.6}
    if op == "act_backward":
        act = rng.random() < 0.8  # without an activation dZ is dY: the bias's gradient is all there is
        return {"op": op, "M": _log(rng, 1, 4608, 1), "N": _log(rng, 64, 12288, 8), "act": act,
                "dbias": not act or rng.random() < 0.8}
    path = rng.choice(["sparse", "sparse", "dense", "w4"])
    act = rng.random() < 0.4
    case = {"op": op, "path": path, "bias": rng.random() < 0.7, "R": rng.random() < 0.8, "act": act}
    if path == "w4":
        g = rng.choice([32, 64, 128])
        case.update(M=rng.randint(1, 32), N=_log(rng, 512, 9216, 8), K=_log(rng, 512, 4096, max(g, 64)), group=g,
                    r=rng.choice([0, 16, 64]), Z=False)
    else:
        case.update(M=_log(rng, 1, 4608, 1), N=_log(rng, 64, 9216, 8), K=_log(rng, 64, 4096, 64),
                    r=rng.choice([0, 16, 64, 64, 144]), Z=rng.random() < 0.4)
    return case


# ---------------------------------------------------------------------------
# inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std


def _stream(g, M, K):
    """Residual stream: rows of their own scale and offset, a few channels of large values."""
    z = _normal(g, (M, K), 1.0) * (0.5 + torch.rand((M, 1), generator=g, device=DEV)) + _normal(g, (M, 1), 0.2)
    loud = torch.rand((1, K), generator=g, device=DEV) < 0.005
    return torch.where(loud, z * 12.0, z).to(BF)


def _activations(g, M, K, gelu):
    """GELU of N(-0.5, 1), or a heavy-tailed mixture (8 % N(0, 1), the rest N(0, 0.05))."""
    z = _normal(g, (M, K), 1.0)
    if gelu:
        return _gelu(z - 0.5).to(BF)
    large = torch.rand((M, K), generator=g, device=DEV) < 0.08
    return torch.where(large, z, z * 0.05).to(BF)


# the place of each nibble of a 32-bit word of 8 consecutive values: low to
# high they hold k = 0, 2, 4, 6, 1, 3, 5, 7
_NIBBLES = [0, 2, 4, 6, 1, 3, 5, 7]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    M = case["M"]
    if op == "act_backward":
        N = case["N"]
        s["dY"] = _normal(g, (M, N), 1e-3).to(BF)
        s["Z"] = (_normal(g, (M, N), 1.0) - 0.5).to(BF)
        return s
    K = case["K"]
    if op in ("layer_norm", "layer_norm_backward"):
        s["X"] = _stream(g, M, K)
        s["weight"] = (1.0 + _normal(g, (K,), 0.2)).to(BF) if case["affine"] else None
        s["bias"] = _normal(g, (K,), 0.1).to(BF) if case["affine"] else None
        if op == "layer_norm_backward":
            x = s["X"].double()
            mean = x.mean(-1)
            var = (x - mean[:, None]).square().mean(-1)
            s["mean"], s["rstd"] = mean.float(), (var + EPS).rsqrt().float()
            s["dY"] = _normal(g, (M, K), 1e-3).to(BF)
            s["dR"] = _normal(g, (M, K), 1e-3).to(BF) if case["dR"] else None
        return s
    N, r = case["N"], case["r"]
    s["X"] = _activations(g, M, K, K > N)
    s["bias"] = _normal(g, (N,), 0.02).to(BF) if case["bias"] else None
    s["A"] = _normal(g, (r, K), 0.01).to(BF) if r else None
    s["B"] = _normal(g, (N, r), 0.01).to(BF) if r else None
    s["R"] = _normal(g, (M, N), 1.0).to(BF) if case["R"] else None
    if case["path"] == "w4":
        q = torch.randint(0, 16, (N, K), generator=g, device=DEV, dtype=torch.uint8)
        n = q.view(N, K // 8, 8)[:, :, _NIBBLES].reshape(N, K // 2, 2)
        s["Wq"] = (n[..., 0] | (n[..., 1] << 4)).contiguous()
        spread = 0.8 + 0.4 * torch.rand((K // case["group"], N), generator=g, device=DEV)
        s["scales"] = (spread / (4.6 * math.sqrt(K))).to(BF)
    else:
        s["W"] = _normal(g, (N, K), 1.0 / math.sqrt(K)).to(BF)
    return s


# ---------------------------------------------------------------------------
# plain forms


_C = math.sqrt(2.0 / math.pi)


def _gelu(v):
    return 0.5 * v * (1.0 + torch.tanh(_C * (v + 0.044715 * v * v * v)))


def _gelu_slope(v):
    t = torch.tanh(_C * (v + 0.044715 * v * v * v))
    return 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * _C * (1.0 + 3 * 0.044715 * v * v)


def _selected(x):
    """S(x) in 32 bits: of each 4 the two of largest magnitude, ties to the lower index, times sum|x| / sum|kept|."""
    ax = x.abs()
    a = ax.view(x.shape[0], -1, 4)
    lower = torch.ones(4, 4, dtype=torch.bool, device=x.device).tril(-1)  # [i, j]: j < i
    keep = torch.empty_like(a, dtype=torch.bool)
    for i in range(4):
        ahead = (a > a[..., i:i + 1]) | ((a == a[..., i:i + 1]) & lower[i])
        keep[..., i] = ahead.sum(-1) < 2
    keep = keep.view_as(x)
    kept = (ax * keep).sum(-1, keepdim=True)
    comp = torch.where(kept > 0, ax.sum(-1, keepdim=True) / kept.clamp_min(1e-37), torch.ones_like(kept))
    return x * keep * comp


def _w4_weight(Wq, scales):
    N, K2 = Wq.shape
    n = torch.stack([Wq & 15, Wq >> 4], dim=-1).view(N, K2 // 4, 8)
    q = n[:, :, [_NIBBLES.index(k) for k in range(8)]].reshape(N, scales.shape[0], -1)
    return ((q.float() - 8.0) * scales.t().float()[..., None]).view(N, 2 * K2)


def _plain(s):
    case, op = s["case"], s["op"]
    if op == "layer_norm":
        x = s["X"].float()
        mean = x.mean(-1, keepdim=True)
        d = x - mean
        rstd = ((d * d).mean(-1, keepdim=True) + EPS).rsqrt()
        y = d * rstd
        if s["weight"] is not None:
            y = y * s["weight"].float() + s["bias"].float()
        return {"Y": y.to(BF), "mean": mean[:, 0], "rstd": rstd[:, 0]} if case["stats"] else {"Y": y.to(BF)}
    if op == "layer_norm_backward":
        dy, x = s["dY"].float(), s["X"].float()
        xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
        g = dy * s["weight"].float() if s["weight"] is not None else dy
        dx = s["rstd"][:, None] * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
        if s["dR"] is not None:
            dx = dx + s["dR"].float()
        if s["weight"] is None:
            return {"dX": dx.to(BF)}
        return {"dX": dx.to(BF), "dweight": (dy * xh).sum(0).to(BF), "dbias": dy.sum(0).to(BF)}
    if op == "act_backward":
        if not case["act"]:
            return {"dbias": s["dY"].float().sum(0).to(BF)}
        dz = s["dY"].float() * _gelu_slope(s["Z"].float())
        return {"dZ": dz.to(BF), "dbias": dz.sum(0).to(BF)} if case["dbias"] else {"dZ": dz.to(BF)}
    x = s["X"].float()
    if case["path"] == "w4":
        p = x @ _w4_weight(s["Wq"], s["scales"]).t()
    else:
        p = (_selected(x) if case["path"] == "sparse" else x) @ s["W"].float().t()
    if s["A"] is not None:
        p = p + (x @ s["A"].float().t()) @ s["B"].float().t()
    if s["bias"] is not None:
        p = p + s["bias"].float()
    y = _gelu(p) if case["act"] else p
    if s["R"] is not None:
        y = y + s["R"].float()
    return {"Y": y.to(BF), "Z": p.to(BF)} if case["Z"] else {"Y": y.to(BF)}


# ---------------------------------------------------------------------------
# the framework's calls


def _own(s):
    from activation_sparse_gemm_lynx_b200 import lynx

    case, op = s["case"], s["op"]
    if op == "layer_norm":
        if not case["stats"]:
            return {"Y": lynx.lynx_layer_norm(s["X"], s["weight"], s["bias"], eps=EPS)}
        Y, mean, rstd = lynx.lynx_layer_norm(s["X"], s["weight"], s["bias"], eps=EPS, want_stats=True)
        return {"Y": Y, "mean": mean, "rstd": rstd}
    if op == "layer_norm_backward":
        affine = s["weight"] is not None
        dX, dweight, dbias = lynx.lynx_layer_norm_backward(s["dY"], s["X"], s["mean"], s["rstd"], s["weight"],
                                                           dR=s["dR"], want_weight=affine, want_bias=affine)
        return {"dX": dX, "dweight": dweight, "dbias": dbias} if affine else {"dX": dX}
    act = lynx.LYNX_ACT_GELU_TANH if case["act"] else lynx.LYNX_ACT_NONE
    if op == "act_backward":
        dZ, dbias = lynx.lynx_act_backward(s["dY"], s["Z"] if case["act"] else None, act=act, want_bias=case["dbias"])
        if not case["act"]:
            return {"dbias": dbias}
        return {"dZ": dZ, "dbias": dbias} if case["dbias"] else {"dZ": dZ}
    if case["path"] == "w4":
        return {"Y": lynx.lynx_linear_w4_residual(s["X"], s["Wq"], s["scales"], None, s["bias"], s["A"], s["B"],
                                                  R=s["R"], act=act)}
    Y, Z = lynx.lynx_linear_residual(s["X"], s["W"], s["bias"], s["A"], s["B"], R=s["R"],
                                     skip_sparsify=case["path"] == "dense", act=act, want_Z=case["Z"])
    return {"Y": Y, "Z": Z} if case["Z"] else {"Y": Y}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# work


def work(case):
    op, M = case["op"], case["M"]
    if op == "act_backward":
        N = case["N"]
        return {"bytes": 2 * M * N * (3 if case["act"] else 1) + (2 * N if case["dbias"] else 0),
                "flops": (16 if case["act"] else 1) * M * N}
    K = case["K"]
    if op == "layer_norm":
        return {"bytes": 4 * M * K + (4 * K if case["affine"] else 0) + (8 * M if case["stats"] else 0),
                "flops": 8 * M * K}
    if op == "layer_norm_backward":
        return {"bytes": 2 * M * K * (4 if case["dR"] else 3) + 8 * M + (6 * K if case["affine"] else 0),
                "flops": 16 * M * K}
    N, r = case["N"], case["r"]
    ends = 2 * M * K + 2 * M * N * (1 + case["R"] + case["Z"]) + 2 * r * (N + K) + (2 * N if case["bias"] else 0)
    branch = 2 * M * r * (N + K)
    if case["path"] == "w4":
        return {"bytes": ends + N * K // 2 + 2 * N * (K // case["group"]), "flops": 2 * M * N * K + branch}
    # the sparse product multiplies the kept half of X
    return {"bytes": ends + 2 * N * K, "flops": (1 if case["path"] == "sparse" else 2) * M * N * K + branch}


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def _exact_selected(X):
    M, K = X.shape
    top = torch.sort(X.abs().reshape(M, -1, 4), dim=2, descending=True, stable=True).indices[..., :2]
    m = torch.zeros(M, K // 4, 4, dtype=torch.float64, device=DEV).scatter_(2, top, 1.0).reshape(M, K)
    everything, held = X.abs().sum(dim=1), (m * X.abs()).sum(dim=1)
    return m * X * torch.where(held > 0, everything / held, torch.ones_like(held))[:, None]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "act_backward":
        if not case["act"]:
            return {"dbias": torch.einsum("mn->n", st["dY"].double())}
        # gelu(z) = z sig(a), a = 2 sqrt(2 / pi) (z + 0.044715 z^3); gelu' = sig + z sig (1 - sig) a'
        z = st["Z"].double()
        c = math.sqrt(8 / math.pi)
        sig = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        dZ = st["dY"].double() * (sig + z * sig * (1 - sig) * c * (1 + 0.134145 * z ** 2))
        return {"dZ": dZ, "dbias": torch.einsum("mn->n", dZ)} if case["dbias"] else {"dZ": dZ}
    if op == "layer_norm":
        x = st["X"].double()
        rstd = 1 / torch.sqrt(torch.var(x, dim=1, unbiased=False) + EPS)
        mean = torch.einsum("mk->m", x) / x.shape[1]
        y = (x - mean[:, None]) * rstd[:, None]
        if st["weight"] is not None:
            y = torch.addcmul(st["bias"].double(), y, st["weight"].double())
        return {"Y": y, "mean": mean, "rstd": rstd} if case["stats"] else {"Y": y}
    if op == "layer_norm_backward":
        K = case["K"]
        w = st["weight"].double() if st["weight"] is not None else torch.ones(K, dtype=torch.float64, device=DEV)
        rstd, dY = st["rstd"].double(), st["dY"].double()
        n = torch.einsum("mk,m->mk", st["X"].double() - st["mean"].double().unsqueeze(1), rstd)
        a = torch.einsum("mk,k->m", dY, w) / K
        b = torch.einsum("mk,k,mk->m", dY, w, n) / K
        dX = (dY * w - a.unsqueeze(1) - n * b.unsqueeze(1)) * rstd.unsqueeze(1)
        if st["dR"] is not None:
            dX += st["dR"].double()
        if st["weight"] is None:
            return {"dX": dX}
        return {"dX": dX, "dweight": torch.einsum("mk,mk->k", dY, n), "dbias": torch.einsum("mk->k", dY)}
    X = st["X"].double()
    if case["path"] == "w4":
        N, K = st["Wq"].shape[0], 2 * st["Wq"].shape[1]
        word = st["Wq"].reshape(N, K // 8, 4).long()
        word = word[..., 0] + (word[..., 1] << 8) + (word[..., 2] << 16) + (word[..., 3] << 24)
        place = torch.tensor([0, 4, 1, 5, 2, 6, 3, 7], device=DEV)  # the nibble of k = 0..7
        q = ((word[..., None] >> (4 * place)) & 15).reshape(N, K).double()
        W = (q - 8) * st["scales"].double().t().repeat_interleave(case["group"], dim=1)
        P = torch.einsum("mk,nk->mn", X, W)
    else:
        S = _exact_selected(X) if case["path"] == "sparse" else X
        P = torch.einsum("mk,nk->mn", S, st["W"].double())
    if st["A"] is not None:
        P += torch.einsum("mr,nr->mn", torch.einsum("mk,rk->mr", X, st["A"].double()), st["B"].double())
    if st["bias"] is not None:
        P += st["bias"].double()
    Y = P * torch.sigmoid(math.sqrt(8 / math.pi) * (P + 0.044715 * P ** 3)) if case["act"] else P
    if st["R"] is not None:
        Y = Y + st["R"].double()
    return {"Y": Y, "Z": P} if case["Z"] else {"Y": Y}
