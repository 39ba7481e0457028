"""Layer norm, the residual epilogue and the activation's gradient at the ends of their ranges."""
import pytest
import torch

from activation_sparse_gemm_lynx_b200 import lynx

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def normal(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


@pytest.mark.parametrize("M,N", [(300, 1000), (4608, 256)])  # a cluster's sums, and sums through the workspace
def test_an_infinite_z_has_no_slope(M, N):
    """GELU's derivative is NaN at either infinity by its formula (and GELU of -inf is NaN), so a row that
    diverged does not send finite gradients back.  Everything else keeps its bits."""
    dY, Z = normal((M, N), 1), normal((M, N), 2)
    Z[0, 0], Z[5, 1], Z[M - 1, N - 2], Z[7, 64] = 3e38, -3e38, -16.0, 16.0  # finite: 0 or 1
    want, wb = lynx.lynx_act_backward(dY, Z)
    assert torch.isfinite(want).all() and float(want[0, 0]) == float(dY[0, 0]) and float(want[5, 1]) == 0.0
    places = [(0, 8, "inf"), (0, 9, "-inf"), (M // 2, 63, "-inf"), (M - 1, N - 1, "inf"), (3, 200, "nan")]
    bad = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    for m, n, v in places:
        Z[m, n] = float(v)
        bad[m, n] = True
    dZ, db = lynx.lynx_act_backward(dY, Z)
    assert torch.isnan(dZ[bad]).all() and torch.equal(dZ[~bad], want[~bad])
    cols = bad.any(0)
    assert torch.isnan(db[cols]).all() and torch.equal(db[~cols], wb[~cols])


@pytest.mark.parametrize("K", [56, 104, 328, 448, 1000, 1920, 4032, 4224, 8560, 32760])  # one row a warp to one a block
def test_a_constant_row_has_no_variance(K):
    """K c has at most 15 + 8 bits, so the row's sum is exact and its mean is c itself: Y is the bias, bit for bit,
    however far from zero the row lies (K's reciprocal is not exact, and c K (1 / K) is not c for these)."""
    values = torch.tensor([3.0, 251.0, -100.0, 30080.0, 2.0 ** 100, -1.0078125, 0.0], device="cuda")
    X = values[:, None].expand(-1, K).to(BF).contiguous()
    bias = normal((K,), 1)
    Y, mean, rstd = lynx.lynx_layer_norm(X, normal((K,), 2), bias, eps=1e-6, want_stats=True)
    assert torch.equal(mean, X[:, 0].float())
    assert torch.equal(Y, bias.expand_as(Y))
    assert torch.allclose(rstd, torch.full_like(rstd, 1e3), rtol=1e-5)
    assert torch.isnan(lynx.lynx_layer_norm(X, eps=0.0)).all()


def bits(t):
    return t.view(torch.int16)


@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (300, 1000, 576), (1300, 2056, 256)])  # 1-CTA tiles, CTA pairs
def test_a_negative_zero_keeps_its_sign(M, N, K, skip):
    """GELU of values below about -10 is -0.  Without a residual nothing is added to it: with Z the bits of Y are
    those without."""
    X, W, bias = normal((M, K), 1), normal((N, K), 2, K ** -0.5), normal((N,), 3)
    bias[::5] = -40.0
    want = lynx.lynx_linear_act(X, W, bias, act=lynx.LYNX_ACT_GELU_TANH, skip_sparsify=skip)
    assert (bits(want) == -32768).any()
    Y, Z = lynx.lynx_linear_residual(X, W, bias, act=lynx.LYNX_ACT_GELU_TANH, skip_sparsify=skip, want_Z=True)
    assert torch.equal(bits(Y), bits(want))
    # a residual of -0 leaves it, one of +0 does not
    for zero, sign in ((-0.0, -32768), (0.0, 0)):
        R = torch.full((M, N), zero, dtype=BF, device="cuda")
        Y, _ = lynx.lynx_linear_residual(X, W, bias, R=R, act=lynx.LYNX_ACT_GELU_TANH, skip_sparsify=skip)
        assert torch.all(bits(Y)[bits(want) == -32768] == sign)
