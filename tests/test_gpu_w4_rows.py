"""What include/lynx.h promises about a token's row: at equal M its bits do not depend on
the other rows; between different M only the order of fp32 sums changes."""
import pytest
import torch

from activation_sparse_gemm_lynx_b200 import lynx

import adapter_oracle as ao
from test_gpu_w4 import normal, w4_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,K,group,r", [(264, 640, 64, 0), (4104, 1024, 128, 64), (12288, 512, 32, 64)])
def test_a_tokens_row(N, K, group, r):
    torch.cuda.set_device(0)
    Wq, sc, ze, W = w4_case(N + K, N, K, group, True)
    A, B = (normal(3, r, K, std=0.02), normal(4, N, r, std=0.2)) if r else (None, None)
    token, bias = normal(5, 1, K), normal(6, N)
    ref, tol = ao.linear_w4(token, W, bias, A, B)
    for M in (1, 2, 8, 9, 16, 17, 32):
        rows = []
        for seed, at in ((10, 0), (11, 0), (12, M - 1)):
            X = normal(seed, M, K, std=10.0 ** (seed - 11))
            X[at] = token[0]
            rows.append(lynx.lynx_linear_w4(X, Wq, sc, ze, bias, A, B)[at])
        assert torch.equal(rows[0], rows[1])  # the same place, other rows
        assert torch.equal(rows[0], rows[2])  # another place
        assert bool(((rows[0].double() - ref[0]).abs() <= tol[0]).all())
