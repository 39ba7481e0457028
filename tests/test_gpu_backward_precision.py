"""The adapter's gradients in the norm: they are off by the rounding of the results
alone, and what lies in the last, ragged block of a dimension counts."""
import pytest
import torch

from activation_sparse_gemm_lynx_b200 import lynx

import adapter_oracle as ao
from norms import rounded_once
from test_gpu_w4 import DEV, normal

pytestmark = pytest.mark.gpu
FORMATS = [lynx.LYNX_CKPT8_INT8, lynx.LYNX_CKPT8_E4M3]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    torch.cuda.set_device(0)
    lynx.library()
    yield
    st, code = lynx.lynx_check_error()
    assert st == lynx.LYNX_OK, (st, code)


def gradients(X, dY, A, B, fmt):
    q, e = lynx.lynx_ckpt8_store(X, fmt)
    x = ao.ckpt8_values(q.float().double(), e.long(), fmt == lynx.LYNX_CKPT8_INT8)
    dA, dB, dT = lynx.lynx_lora_backward(dY, q, e, A, B)
    return {"dT": dT, "dB": dB, "dA": dA}, ao.lora_backward(dY, x, A, B)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K,r", [(300, 1000, 576, 16), (2049, 72, 64, 80), (1025, 2056, 128, 192),
                                     (257, 136, 320, 208), (1000, 640, 256, 256), (300, 4104, 320, 256),
                                     (129, 520, 1088, 144), (4608, 1032, 512, 64), (70, 4096, 2048, 240),
                                     (1500, 2056, 4096, 112)])
def test_only_the_results_are_rounded(M, N, K, r, fmt):
    X = normal(M + K, M, K)
    X = torch.where(normal(M, M, K).float() < -1.4, X, X * 0.05)
    dY, A, B = normal(2, M, N, std=1e-3), normal(3, r, K, std=K ** -0.5), normal(4, N, r, std=N ** -0.5)
    got, ref = gradients(X, dY, A, B, fmt)
    for name in got:
        rounded_once(got[name], ref[name][0])


@pytest.mark.parametrize("M,N,K,r", [(2049, 72, 64, 80), (129, 1032, 4160, 64), (300, 264, 192, 256), (1, 8, 64, 16)])
@pytest.mark.parametrize("where", ["rows", "outputs", "columns", "rank"])
def test_the_last_block_counts(where, M, N, K, r):
    """All is zero but the last, ragged block of one dimension."""
    X, dY = normal(1, M, K), normal(2, M, N, std=1e-3)
    A, B = normal(3, r, K, std=K ** -0.5), normal(4, N, r, std=N ** -0.5)

    def last(t, dim, step):
        n = t.shape[dim]
        t.narrow(dim, 0, (n - 1) // step * step).zero_()

    if where == "rows":
        last(X, 0, 128)
    elif where == "outputs":
        last(dY, 1, 128)
    elif where == "columns":
        last(X, 1, 128)
    else:
        last(A, 0, 64)
        last(B, 1, 64)
    got, ref = gradients(X, dY, A, B, lynx.LYNX_CKPT8_INT8)
    for name in got:
        value, tol = ref[name]
        assert bool(value.any())
        assert bool(((got[name].double() - value).abs() <= tol).all())
        if value.count_nonzero() >= 500:
            rounded_once(got[name], value)


def test_an_infinite_gradient_stays_one():
    """Where a partial product overflows, the sum of its two halves is still infinite."""
    M, N, K, r = 2, 64, 64, 16
    X = torch.full((M, K), 1.0, dtype=torch.bfloat16, device=DEV)
    dY = torch.full((M, N), 3.0e38, dtype=torch.bfloat16, device=DEV)
    A, B = torch.ones(r, K, dtype=torch.bfloat16, device=DEV), torch.ones(N, r, dtype=torch.bfloat16, device=DEV)
    dA, dB, dT = lynx.lynx_lora_backward(dY, *lynx.lynx_ckpt8_store(X), A, B)
    for t in (dA, dB, dT):
        assert bool((t == float("inf")).all())
