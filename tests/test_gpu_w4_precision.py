"""The few-token layer in the norm of each output row: nothing is rounded before Y."""
import pytest
import torch

from activation_sparse_gemm_lynx_b200 import lynx

import adapter_oracle as ao
from norms import rounded_once
from test_gpu_w4 import DEV, normal, w4_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("zp", [False, True])
@pytest.mark.parametrize("M,N,K,group,r", [(1, 12288, 4096, 128, 64), (3, 1024, 16384, 128, 256), (8, 520, 576, 64, 16),
                                           (16, 1000, 1088, 64, 256), (17, 4104, 1088, 32, 0), (32, 4104, 512, 128, 64),
                                           (5, 12296, 256, 64, 16), (2, 640, 12288, 32, 48)])
def test_each_row_is_rounded_once(M, N, K, group, r, zp):
    """A weight rounded to bf16 (s (q - z) has up to 13 bits) would add as much again as Y's
    rounding, 1.41 for 1.1."""
    torch.cuda.set_device(0)
    Wq, sc, ze, W = w4_case(N + K, N, K, group, zp)
    X = normal(1, M, K)
    A, B = (normal(3, r, K, std=0.02), normal(4, N, r, std=0.2)) if r else (None, None)
    ref, _ = ao.linear_w4(X, W, None, A, B)
    rounded_once(lynx.lynx_linear_w4(X, Wq, sc, ze, None, A, B), ref, dim=1)


@pytest.mark.parametrize("how", ["zero", "cancels"])
@pytest.mark.parametrize("M,N,K,r", [(1, 1000, 16384, 256), (9, 4104, 512, 64), (32, 520, 1088, 16), (3, 12288, 4096, 144)])
def test_the_branch_alone(M, N, K, r, how):
    """Y = T B^T where the weight is zero, and where X W^T cancels: T's precision shows.  One
    bf16 for T would be off by 1.41 for 1.1 of Y's rounding."""
    torch.cuda.set_device(0)
    Wq, sc, ze, W = w4_case(N + K, N, K, 32, True)
    X, A, B = normal(1, M, K), normal(3, r, K, std=0.02), normal(4, N, r, std=0.2)
    if how == "zero":
        sc, W = torch.zeros_like(sc), torch.zeros_like(W)
    else:
        # every k of an even group is taken back by the same place of the next one: the
        # group sums are equal and opposite, in fp32 too, when they are formed in one order
        pairs = K // 64
        q = torch.randint(0, 16, (N, pairs, 1, 32), generator=torch.Generator(device=DEV).manual_seed(7), device=DEV)
        q = q.expand(N, pairs, 2, 32).reshape(N, K)
        sc = torch.full_like(sc, 2.0 ** -6)
        ze = torch.full_like(ze, 5)
        Wq = ao.w4_pack(q)
        W = (q.double() - 5) * 2.0 ** -6
        X = X.reshape(M, pairs, 2, 32).clone()
        X[:, :, 1] = -X[:, :, 0]
        X = X.reshape(M, K).contiguous()
        assert float((X.double() @ W.t()).abs().max()) < 1e-9
    ref, _ = ao.linear_w4(X, W, None, A, B)
    Y = lynx.lynx_linear_w4(X, Wq, sc, ze, None, A, B)
    if how == "zero":
        rounded_once(Y, ref, dim=1)
        return
    # A pair's two sums are added one after the other, so the running sum is at most one group's
    # |x| |w| and each of the two additions loses at most 2^-24 of it.
    off = (Y.double() - ref).norm(dim=1)
    most = 1.1 * (ref.bfloat16().double() - ref).norm(dim=1) + 2.0 ** -12 * ref.norm(dim=1)
    left = 2.0 ** -23 * (X.double().abs() @ W.abs().t()).norm(dim=1)
    assert bool((off <= most + left).all())
