"""Layers that the CTA pairs take, at ragged sizes and odd ranks, with everything that can be in
their epilogue, against the formulas in 64 bits.  That the pairs did take them shows in the state
words at the end of the workspace (test_gpu_gemm_choice.py).
"""
import random

import pytest
import torch

import bench
import block_oracle as oracle
from activation_sparse_gemm_lynx_b200 import lynx
from test_gpu_gemm_choice import state_words

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
NONE, GELU = lynx.LYNX_ACT_NONE, lynx.LYNX_ACT_GELU_TANH


def normal(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


def layer(M, N, K, r, bias=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn((M, K), generator=g, device="cuda")
    X = torch.where(torch.rand((M, K), generator=g, device="cuda") < 0.08, z, 0.05 * z).to(BF)
    return (X, normal((N, K), seed + 1, K ** -0.5), normal((N,), seed + 2, 0.02) if bias else None,
            normal((r, K), seed + 3, 0.05) if r else None, normal((N, r), seed + 4, 0.05) if r else None)


def check(M, N, K, r, skip, act, with_r, with_z, bias=True, fill=0x5A5A5A5A, seed=0):
    """One layer in buffers with room behind them, its workspace filled with `fill` before."""
    assert bench.uses_pair_gemm(M, N, K, sparse=not skip, r=r)
    X, W, bias, A, B = layer(M, N, K, r, bias, seed)
    R = normal((M, N), seed + 9) if with_r else None
    room = torch.full((2, M + 3, N), 7.0, dtype=BF, device="cuda")
    ws = None
    if r or not skip:
        ws = torch.empty(lynx.lynx_workspace_bytes(M, N, K, r), dtype=torch.uint8, device="cuda")
        ws.view(torch.int32).fill_(fill)
    Y, Z = lynx.lynx_linear_residual(X, W, bias, A, B, R=R, skip_sparsify=skip, act=act, Y=room[0, :M],
                                     Z=room[1, :M] if with_z else None, workspace=ws)
    assert lynx.lynx_check_error() == (lynx.LYNX_OK, 0)
    assert torch.all(room[:, M:] == 7.0) and (with_z or torch.all(room[1] == 7.0))
    want = oracle.linear_residual(X, W, bias, A, B, R, skip, act == GELU)
    oracle.check(Y, want["Y"], "Y")
    if with_z:
        oracle.check(Z, want["Z"], "Z")
    if ws is not None:
        assert torch.all(state_words(ws, M) == 2)  # each 32 rows joined, once
    return (X, W, bias, A, B), R, Y, Z


# N on 32 bytes and on 16, one more column tile of 8 and of 200 columns, a row block of 1 and of 20 rows
SHAPES = [(1300, 2056, 256, 48), (1537, 2064, 384, 144), (1300, 2120, 128, 0)]
SPARSE = [(300, 520, 2176, 16), (129, 264, 2304, 256), (1000, 2304, 1792, 32)]


@pytest.mark.parametrize("act", [NONE, GELU])
@pytest.mark.parametrize("with_r,with_z", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("M,N,K,r,skip", [(*s, False) for s in SHAPES + SPARSE] + [(*s, True) for s in SHAPES])
def test_epilogues(M, N, K, r, skip, with_r, with_z, act):
    args, R, Y, Z = check(M, N, K, r, skip, act, with_r, with_z, seed=M)
    if not with_r:  # what was there before is the same without Z, bit for bit
        was = lynx.lynx_linear_act(*args, act=act, skip_sparsify=skip)
        assert torch.equal(Y.view(torch.int16), was.view(torch.int16))
        if with_z:
            assert torch.equal(Z, lynx.lynx_linear(*args, skip_sparsify=skip))
    elif not with_z:  # in place
        here = R.clone()
        lynx.lynx_linear_residual(*args, R=here, skip_sparsify=skip, act=act, Y=here)
        assert torch.equal(here, Y)


def draw(i):
    rng = random.Random(20261209 + i)
    r = rng.choice([0, 16, 32, 48, 64, 96, 128, 256])
    family = i % 4
    skip = family in (0, 1) and rng.random() < 0.4
    if family == 0:
        M, N, K = rng.randint(1200, 2000), 8 * rng.randint(188, 330), 128 * rng.randint(1, 7)
    elif family == 1:  # two row blocks, many columns
        M, N, K = rng.randint(129, 256), 8 * rng.randint(1200, 1600), 128 * rng.randint(1, 5)
    elif family == 2:
        M, N, K = rng.randint(129, 700), 8 * rng.randint(32, 190), 128 * rng.randint(17, 32)
    else:
        r = rng.choice([0, 16, 32])
        M, N, K = rng.randint(900, 1024), 8 * rng.randint(160, 290), 128 * rng.randint(13, 16)
    return dict(M=M, N=N, K=K, r=r, skip=skip, act=rng.choice([NONE, GELU]), with_r=rng.random() < 0.5,
                with_z=rng.random() < 0.5, bias=rng.random() < 0.7, fill=rng.choice([2, -1, 1, 0x5A5A5A5A]), seed=100 + i)


@pytest.mark.parametrize("i", range(60))
def test_drawn_layers(i):
    c = draw(i)
    (X, W, bias, A, B), _, _, _ = check(**c)
    # the layer's two halves on two streams: the bits of the whole
    act, skip, r = c["act"], c["skip"], c["r"]
    Y = lynx.lynx_linear_act(X, W, bias, A, B, skip_sparsify=skip, act=act)
    ws = torch.empty(lynx.lynx_workspace_bytes(c["M"], c["N"], c["K"], r or 64), dtype=torch.uint8, device="cuda")
    ws.view(torch.int32).fill_(c["fill"])
    Y2 = torch.zeros_like(Y)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    lynx.lynx_linear_begin(X, W, bias, A, B, skip_sparsify=skip, act=act, Y=Y2, workspace=ws, stream=s1)
    s2.wait_stream(s1)
    lynx.lynx_linear_finish(X, W, bias, A, B, skip_sparsify=skip, act=act, Y=Y2, workspace=ws, stream=s2)
    torch.cuda.synchronize()
    assert all(lynx.lynx_check_error(s) == (lynx.LYNX_OK, 0) for s in (None, s1, s2))
    assert torch.equal(Y.view(torch.int16), Y2.view(torch.int16)), c


def test_either_kernel_gives_the_same_bits_sparse_and_with_an_adapter():
    """Row blocks of one S(X) alone, where the 1-CTA kernel takes them with tiles of 32 to 128 columns."""
    M, N, K, r = 2304, 2048, 512, 48
    X, W, bias, _, B = layer(M, N, K, r, seed=5)
    T = normal((M, r), 11)
    vals, meta, _ = lynx.lynx_sparsify(X)
    whole = lynx.lynx_sparse_gemm(vals, meta, W, bias, T=T, B=B)
    plain = lynx.lynx_sparse_gemm(vals, meta, W)
    assert bench.uses_pair_gemm(M, N, K)
    block = meta.numel() * 256 // M  # of 256 rows
    for r0, r1 in ((0, 256), (256, 300), (512, 1536), (1024, 2000), (2048, 2049)):
        assert not bench.uses_pair_gemm(r1 - r0, N, K)
        m = meta[r0 // 256 * block:].contiguous()
        assert torch.equal(lynx.lynx_sparse_gemm(vals[r0:r1], m, W, bias, T=T[r0:r1], B=B), whole[r0:r1]), (r0, r1)
        assert torch.equal(lynx.lynx_sparse_gemm(vals[r0:r1], m, W), plain[r0:r1]), (r0, r1)
    assert lynx.lynx_check_error() == (lynx.LYNX_OK, 0)


@pytest.mark.parametrize("M,N,K", [(1300, 2056, 256), (300, 520, 2176)])
def test_two_host_threads_on_the_pairs(M, N, K):
    """Both at once, each on its own stream with its own buffers: what each gives alone."""
    import threading

    args = layer(M, N, K, 16, seed=8)
    R = normal((M, N), 9)
    want = lynx.lynx_linear_residual(*args, R=R, act=GELU, want_Z=True)
    torch.cuda.synchronize()
    bad = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = lynx.lynx_linear_residual(*args, R=R, act=GELU, want_Z=True)
            torch.cuda.current_stream().synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want)) or lynx.lynx_check_error()[0] != lynx.LYNX_OK:
                bad.append("different")

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
