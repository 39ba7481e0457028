"""The adapter's T of the few-token layer at the end of fp32's range."""
import pytest
import torch

from activation_sparse_gemm_lynx_b200 import lynx

import adapter_oracle as ao
from test_gpu_w4 import DEV

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def branch(M, N, K, r, x, a, b):
    """The layer with a weight of zeros: Y = T B^T.  x, a: the first values of each row."""
    torch.cuda.set_device(0)
    X, A = torch.zeros(M, K, dtype=BF, device=DEV), torch.zeros(r, K, dtype=BF, device=DEV)
    X[:, :len(x)] = torch.tensor(x, device=DEV).to(BF)
    A[:, :len(a)] = torch.tensor(a, device=DEV).to(BF)
    B = torch.full((N, r), b, dtype=BF, device=DEV)
    Wq = torch.full((N, K // 2), 0x88, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(K // 32, N, dtype=BF, device=DEV)
    Y = lynx.lynx_linear_w4(X, Wq, scales, None, None, A, B)
    return Y, ao.linear_w4(X, torch.zeros(N, K, dtype=torch.float64, device=DEV), None, A, B)


@pytest.mark.parametrize("M", [1, 9, 32])
def test_an_infinite_branch_stays_one(M):
    """T overflows fp32; every product with it has one sign."""
    for sign in (1.0, -1.0):
        Y, _ = branch(M, 264, 128, 32, [3.0e38, 3.0e38], [1.0, 1.0], sign * 1e-3)
        assert bool((Y == sign * float("inf")).all())


@pytest.mark.parametrize("M", [1, 9, 32])
def test_the_largest_finite_branch(M):
    """T = 3.3975e38, between the largest bf16 with half a step and the largest fp32."""
    x, a = [3.3895e38, 8.0e35], [1.0, 1.0]
    Y, (ref, tol) = branch(M, 264, 128, 16, x, a, 2.0 ** -8)
    T = sum(float(torch.tensor(v).to(BF)) for v in x)
    assert 3.3962e38 < T < 3.4028e38
    assert bool(torch.isfinite(Y).all()) and bool(((Y.double() - ref).abs() <= tol).all())
