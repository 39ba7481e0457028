"""Layer norm over many rows: a block's threads take one row after another, the next ones on their
way in a ring of shared memory, and the columns' sums go through the workspace.

Against the formulas in 64 bits.  No chain of additions is longer than the 128 that
block_oracle.SUM allows: a column's are 8 rows at most of a group of threads, 8 groups, 148 blocks in
32 ways of 5 and those in 4 of 8; past 8192 columns 34 rows of a thread, 8 threads and the ranges.
"""
import pytest
import torch

import block_oracle as oracle
from activation_sparse_gemm_lynx_b200 import lynx, workloads

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
EPS = 1e-6
HIDDEN = workloads.CONFIGS["mlp_up"].K  # 3 warps a row forward, 6 backward, no branches


def stream(M, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn((M, K), generator=g, device="cuda") * (0.5 + torch.rand((M, 1), generator=g, device="cuda"))
    return (z + 0.2 * torch.randn((M, 1), generator=g, device="cuda")).to(BF)


def normal(shape, seed, mean=0.0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (mean + std * torch.randn(shape, generator=g, device="cuda")).to(BF)


# 2 to 6 rows a group of threads, each count of pieces a thread, with and without branches
@pytest.mark.parametrize("M,K", [(9000, 64), (20000, 264), (12000, 512), (9000, HIDDEN), (3000, 4096), (5000, 1088), (1300, 8200),
                                 (1200, 16384), (700, 32768)])
def test_forward(M, K):
    X, w, b = stream(M, K, M + K), normal((K,), 1, 1.0, 0.2), normal((K,), 2, 0.0, 0.1)
    Y, mean, rstd = lynx.lynx_layer_norm(X, w, b, eps=EPS, want_stats=True)
    want = oracle.layer_norm(X, w, b, EPS)
    oracle.check(Y, want["Y"], "Y")
    oracle.check(mean, want["mean"], "mean")
    oracle.check(rstd, want["rstd"], "rstd")
    # a row is the same whichever rows are before and after it
    for r0, r1 in ((0, 3), (M // 2, M // 2 + 5), (M - 2, M)):
        y, m, s = lynx.lynx_layer_norm(X[r0:r1], w, b, eps=EPS, want_stats=True)
        assert torch.equal(y, Y[r0:r1]) and torch.equal(m, mean[r0:r1]) and torch.equal(s, rstd[r0:r1])


# two, four and eight pieces a thread; one to four stages of the ring (dR is a third of one), each gone
# round more than once; past 8192 columns the sums are a pass of their own, through the workspace from
# 321 rows on
@pytest.mark.parametrize("branch", [True, False])
@pytest.mark.parametrize("M,K", [(9000, 64), (6000, 576), (1500, HIDDEN), (1500, 4096), (700, 8192), (330, 8200), (700, 12288),
                                 (400, 16392), (800, 32768)])
def test_backward(M, K, branch):
    X, dY, w = stream(M, K, M + K), normal((M, K), 1), normal((K,), 1, 1.0, 0.2)
    dR = normal((M, K), 2) if branch else None
    _, mean, rstd = lynx.lynx_layer_norm(X, w, None, eps=EPS, want_stats=True)
    dX, dw, db = lynx.lynx_layer_norm_backward(dY, X, mean, rstd, w, dR=dR)
    want = oracle.layer_norm_backward(dY, X, mean, rstd, w, dR)
    oracle.check(dX, want["dX"], "dX")
    oracle.check(dw, want["dweight"], "dweight")
    oracle.check(db, want["dbias"], "dbias")
    # the rows alone, without the columns' sums: the same bits, the other kernel
    alone, none, none2 = lynx.lynx_layer_norm_backward(dY, X, mean, rstd, w, dR=dR, want_weight=False, want_bias=False)
    assert none is None and none2 is None and torch.equal(alone, dX)
    # one of the two sums, and dX over dR
    here = dR.clone() if branch else None
    same, dw2, _ = lynx.lynx_layer_norm_backward(dY, X, mean, rstd, w, dR=here, dX=here, want_bias=False)
    assert torch.equal(same, dX) and torch.equal(dw2, dw)
    _, _, db2 = lynx.lynx_layer_norm_backward(dY, X, mean, rstd, w, dR=dR, want_weight=False)
    assert torch.equal(db2, db)


@pytest.mark.parametrize("M,K", [(1500, 4096), (700, 12288)])
def test_a_stale_workspace_and_nothing_behind_it(M, K):
    X, dY, w = stream(M, K, 1), normal((M, K), 1), normal((K,), 1, 1.0, 0.2)
    _, mean, rstd = lynx.lynx_layer_norm(X, w, None, eps=EPS, want_stats=True)
    want = lynx.lynx_layer_norm_backward(dY, X, mean, rstd, w)
    need = lynx.lynx_layer_norm_backward_workspace_bytes(M, K)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN
    for _ in range(2):
        for a, b in zip(lynx.lynx_layer_norm_backward(dY, X, mean, rstd, w, workspace=ws), want):
            assert torch.equal(a, b)
    assert torch.all(ws[need:] == 0xFF)
