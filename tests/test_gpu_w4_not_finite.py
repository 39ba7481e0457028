"""Weights that are not finite: their group stands for NaN, as the formula of its scale
says, and no other group is touched."""
import pytest
import torch

from activation_sparse_gemm_lynx_b200 import lynx

import adapter_oracle as ao
from test_gpu_w4 import DEV, normal

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("zp", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_the_group_stands_for_nan(group, zp):
    torch.cuda.set_device(0)
    N, K = 72, 1152
    W = normal(1, N, K, std=0.05)
    clean = W.clone()
    bad = torch.zeros(N, K // group, dtype=torch.bool, device=DEV)
    nan = bad.clone()
    # (row, columns, value): every place of a lane's 8 values, of a packed pair and of a group
    places = [(n, [n * 17 % K], v) for n, v in zip(range(8, 24), [NAN, INF, -INF, -NAN] * 4)]
    places += [(24, list(range(8)), NAN), (25, list(range(group)), NAN), (26, [K - 1], NAN), (27, [0, 1], INF),
               (28, [3, 9], None), (71, [K - 2], -INF)]
    for n, cols, v in places:
        if v is None:  # both infinities in a group
            W[n, 3], W[n, 9] = INF, -INF
        else:
            W[n, cols] = v
        for k in cols:
            bad[n, k // group] = True
            nan[n, k // group] |= v is not None and v != v
    W[29, 5], W[29, 6] = INF, NAN
    bad[29, 0] = nan[29, 0] = True
    Wq, sc, ze = lynx.lynx_w4_quantize(W, group, zp)
    s = sc.t().double()
    assert torch.equal(torch.isnan(s), nan)
    assert torch.equal(torch.isinf(s), bad & ~nan)
    back = lynx.lynx_w4_dequantize(Wq, sc, ze)
    wide = bad.repeat_interleave(group, 1)
    assert torch.equal(torch.isnan(back), wide)
    # q = z in such a group, and everything else is as without it
    q0, s0, z0 = ao.w4_quantize(clean, group, zp)
    z = torch.where(bad, 0.0 if zp else 8.0, z0)
    q = torch.where(wide, z.repeat_interleave(group, 1), q0)
    assert torch.equal(Wq, ao.w4_pack(q))
    if zp:
        assert torch.equal(ze.double(), z.t())
    assert torch.equal(s[~bad], s0[~bad])
    assert torch.equal(back[~wide], ao.w4_values(q0, s0, z0).bfloat16()[~wide])
    # an output is NaN if its row has such a group, and only then
    X = normal(2, 3, K)
    Y = lynx.lynx_linear_w4(X, Wq, sc, ze)
    rows = bad.any(1)
    assert bool(torch.isnan(Y[:, rows]).all())
    ref, tol = ao.linear_w4(X, ao.w4_values(q0, s0, z0))
    assert bool(((Y.double() - ref).abs() <= tol)[:, ~rows].all())
