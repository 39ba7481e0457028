"""The selection gradient at both ends of the range: its row sums are ratios, whatever the
row's magnitude."""
import pytest
import torch

from activation_sparse_gemm_lynx_b200 import lynx

import adapter_oracle as ao
import selection_oracle as so
from test_gpu_w4 import DEV, normal

pytestmark = pytest.mark.gpu
FORMATS = [lynx.LYNX_CKPT8_INT8, lynx.LYNX_CKPT8_E4M3]


def check(X, G, fmt):
    M, K = X.shape
    q, e = lynx.lynx_ckpt8_store(X, fmt)
    x = ao.ckpt8_values(q.float().double(), e.long(), fmt == lynx.LYNX_CKPT8_INT8)
    assert bool(torch.isfinite(x).all())
    # the bounds of the oracles hold at any magnitude; below 2^-126 an absolute one
    ref, tol = ao.sparsify_backward(G, x)
    dX = lynx.lynx_sparsify_backward(G, q, e)
    assert bool(((dX.double() - ref).abs() <= tol).all())
    m = ao.keep(normal(9, M, K).double())
    meta = lynx.lynx_sparsify(normal(9, M, K))[1]
    ref, tol = so.gradient(G, x, m)
    dX = lynx.lynx_sparsify_backward(G, q, e, meta=meta)
    assert bool(((dX.double() - ref).abs() <= tol).all())
    return dX


@pytest.fixture(scope="module", autouse=True)
def _lib():
    torch.cuda.set_device(0)
    lynx.library()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("K", [256, 1088, 12288])
def test_rows_of_every_magnitude(K, fmt):
    """Row i near 2^(i - 131): from subnormal values to where a few of them overflow a sum."""
    M = 256
    scale = torch.exp2(torch.arange(M, device=DEV, dtype=torch.float64) - 131)[:, None]
    X = normal(1, M, K).double().clamp(-3.9, 3.9) * scale
    X = X.clamp(-3.38e38, 3.38e38).bfloat16()
    check(X, normal(2, M, K, std=1e-6), fmt)
    check(X, normal(2, M, K, std=1e4), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("K", [576, 4096, 16448])
def test_blocks_of_many_magnitudes_in_a_row(K, fmt):
    """Exponents that rise, fall, alternate and jump along a row, 200 binades apart."""
    n = K // 32
    t = torch.linspace(-100, 100, n, device=DEV).round().double()
    g = torch.Generator(device=DEV).manual_seed(3)
    orders = [t, t.flip(0), torch.where(torch.arange(n, device=DEV) % 2 == 0, t, -t),
              t[torch.randperm(n, generator=g, device=DEV)], torch.full_like(t, -120.0), torch.zeros_like(t)]
    orders[4][-1] = 100.0  # all but the last block vanish beside it
    orders[5][n // 2] = -130.0
    scale = torch.exp2(torch.stack(orders)).repeat_interleave(32, 1)
    X = (normal(4, len(orders), K).double() * scale).bfloat16()
    check(X, normal(5, len(orders), K, std=1e-3), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_the_largest_gradients(fmt):
    """|G| up to 2^88, which the header names."""
    M, K = 5, 4096
    X = normal(6, M, K)
    G = (normal(7, M, K).float().clamp(-1, 1) * 2.0 ** 88).bfloat16()
    dX = check(X, G, fmt)
    assert bool(torch.isfinite(dX).all())
