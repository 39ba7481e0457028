"""lynx_linear_residual, lynx_linear_w4_residual and lynx_act_backward against the
formulas in 64 bits."""
import pytest
import torch

import block_oracle as oracle
from activation_sparse_gemm_lynx_b200 import lynx

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
NONE, GELU = lynx.LYNX_ACT_NONE, lynx.LYNX_ACT_GELU_TANH


def normal(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


def layer(M, N, K, r, seed=0, bias=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn((M, K), generator=g, device="cuda")
    X = torch.where(torch.rand((M, K), generator=g, device="cuda") < 0.08, z, 0.05 * z).to(BF)
    return (X, normal((N, K), seed + 1, K ** -0.5), normal((N,), seed + 2, 0.02) if bias else None,
            normal((r, K), seed + 3, 0.05) if r else None, normal((N, r), seed + 4, 0.05) if r else None)


# one row and one column tile of either kernel, ragged last tiles, the CTA-pair kernel with and
# without a full tile, K that only the single-CTA kernel takes
SHAPES = [(1, 8, 64, 0), (1, 512, 512, 16), (300, 1000, 576, 16), (129, 256, 128, 0), (257, 264, 256, 16), (256, 512, 512, 64),
          (600, 1288, 384, 144), (130, 2048, 640, 64)]


@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("act", [NONE, GELU])
@pytest.mark.parametrize("M,N,K,r", SHAPES)
def test_layer(M, N, K, r, act, skip):
    X, W, bias, A, B = layer(M, N, K, r, seed=M, bias=N != 264)
    R = normal((M, N), 9)
    Y, Z = lynx.lynx_linear_residual(X, W, bias, A, B, R=R, skip_sparsify=skip, act=act, want_Z=True)
    want = oracle.linear_residual(X, W, bias, A, B, R, skip, act == GELU)
    oracle.check(Y, want["Y"], "Y")
    oracle.check(Z, want["Z"], "Z")
    assert lynx.lynx_check_error() == (lynx.LYNX_OK, 0)


@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("M,N,K,r", [(300, 1000, 576, 16), (600, 1288, 384, 64)])
def test_each_part_alone_is_the_layer_that_was(M, N, K, r, skip):
    X, W, bias, A, B = layer(M, N, K, r, seed=1)
    R = normal((M, N), 9)
    kw = dict(skip_sparsify=skip)
    for act in (NONE, GELU):
        was = lynx.lynx_linear_act(X, W, bias, A, B, act=act, **kw)
        Y, Z = lynx.lynx_linear_residual(X, W, bias, A, B, act=act, **kw)
        assert Z is None and torch.equal(Y, was)
        Y, Z = lynx.lynx_linear_residual(X, W, bias, A, B, act=act, want_Z=True, **kw)
        assert torch.equal(Y, was)
        assert torch.equal(Z, lynx.lynx_linear(X, W, bias, A, B, **kw))
        both, _ = lynx.lynx_linear_residual(X, W, bias, A, B, R=R, act=act, want_Z=True, **kw)
        alone, none = lynx.lynx_linear_residual(X, W, bias, A, B, R=R, act=act, **kw)
        assert none is None and torch.equal(alone, both)
        here = R.clone()  # the stream updated in place
        out, _ = lynx.lynx_linear_residual(X, W, bias, A, B, R=here, act=act, Y=here, **kw)
        assert out.data_ptr() == here.data_ptr() and torch.equal(here, both)


@pytest.mark.parametrize("skip", [False, True])
def test_in_place_over_many_tiles_a_block(skip):
    """More output tiles than blocks, N no multiple of a line: neighbouring tiles share lines of R = Y."""
    M, N, K = 4097, 4104, 128
    X, W, bias, A, B = layer(M, N, K, 16, seed=2)
    R = normal((M, N), 9)
    want, _ = lynx.lynx_linear_residual(X, W, bias, A, B, R=R, skip_sparsify=skip)
    oracle.check(want[-300:], oracle.linear_residual(X[-300:], W, bias, A, B, R[-300:], skip, False)["Y"], "Y")
    here = R.clone()
    lynx.lynx_linear_residual(X, W, bias, A, B, R=here, skip_sparsify=skip, Y=here)
    assert torch.equal(here, want)


def test_a_residual_that_is_not_finite_stays_where_it_is():
    X, W, bias, A, B = layer(200, 512, 256, 0, seed=3)
    R = normal((200, 512), 9)
    R[7, 11], R[150, 300] = float("inf"), float("nan")
    Y, Z = lynx.lynx_linear_residual(X, W, bias, R=R, want_Z=True)
    assert torch.isposinf(Y[7, 11]) and torch.isnan(Y[150, 300]) and torch.isfinite(Z).all()
    R[7, 11] = R[150, 300] = 0
    again, _ = lynx.lynx_linear_residual(X, W, bias, R=R)
    Y[7, 11], Y[150, 300] = again[7, 11], again[150, 300]
    assert torch.equal(Y, again)


@pytest.mark.parametrize("M,N,K", [(37, 1000, 576), (290, 520, 256)])
def test_nothing_behind_the_last_row_is_written(M, N, K):
    X, W, bias, _, _ = layer(M, N, K, 0, seed=4)
    room = torch.full((2, M + 2, N), 7.0, dtype=BF, device="cuda")
    lynx.lynx_linear_residual(X, W, bias, R=normal((M, N), 9), act=GELU, Y=room[0, :M], Z=room[1, :M])
    assert torch.all(room[:, M:] == 7.0)


@pytest.mark.parametrize("M", [1, 5, 17, 32])
@pytest.mark.parametrize("N,K,group,r,act", [(512, 512, 64, 0, NONE), (1000, 576, 32, 16, GELU), (4104, 1024, 128, 64, NONE)])
def test_few_tokens(M, N, K, group, r, act):
    X, W, bias, A, B = layer(M, N, K, r, seed=M)
    Wq, scales, zeros = lynx.lynx_w4_quantize(W, group, zero_points=True)
    R = normal((M, N), 9)
    # the values in 64 bits: lynx_w4_dequantize rounds, the layer does not
    words = Wq.view(N, K // 8, 4).long()
    words = words[..., 0] + (words[..., 1] << 8) + (words[..., 2] << 16) + (words[..., 3] << 24)
    q = ((words[..., None] >> (4 * torch.tensor([0, 4, 1, 5, 2, 6, 3, 7], device="cuda"))) & 15).view(N, K).double()
    Wv = (q - zeros.t().double().repeat_interleave(group, 1)) * scales.t().double().repeat_interleave(group, 1)
    Y = lynx.lynx_linear_w4_residual(X, Wq, scales, zeros, bias, A, B, R=R, act=act)
    oracle.check(Y, oracle.linear_residual(X, Wv, bias, A, B, R, True, act == GELU)["Y"], "Y")
    assert torch.equal(lynx.lynx_linear_w4_residual(X, Wq, scales, zeros, bias, A, B, act=act),
                       lynx.lynx_linear_w4(X, Wq, scales, zeros, bias, A, B, act=act))
    lynx.lynx_linear_w4_residual(X, Wq, scales, zeros, bias, A, B, R=R, act=act, Y=R)
    assert torch.equal(R, Y)


ACT_SHAPES = [(1, 8), (1, 4096), (2, 64), (300, 1000), (33, 136), (257, 576), (1000, 4104), (4608, 256)]


@pytest.mark.parametrize("M,N", ACT_SHAPES)
def test_act_backward(M, N):
    dY, Z = normal((M, N), 1), normal((M, N), 2, 1.5)
    dZ, db = lynx.lynx_act_backward(dY, Z)
    want = oracle.act_backward(dY, Z)
    oracle.check(dZ, want["dZ"], "dZ")
    oracle.check(db, want["dbias"], "dbias")
    alone, none = lynx.lynx_act_backward(dY, Z, want_bias=False)
    assert none is None and torch.equal(alone, dZ)
    same, db2 = lynx.lynx_act_backward(dY, act=NONE)
    assert same.data_ptr() == dY.data_ptr()
    oracle.check(db2, oracle.column_sum(dY.double()), "dbias")
    here = dY.clone()  # in place
    out, again = lynx.lynx_act_backward(here, Z, dZ=here)
    assert out.data_ptr() == here.data_ptr() and torch.equal(here, dZ) and torch.equal(again, db)


def test_the_slope_over_all_of_bf16():
    """Every finite bf16 as Z: the largest and the smallest give slopes of 0, 1/2 and 1, never NaN."""
    Z = torch.arange(65536, device="cuda").to(torch.int32).to(torch.int16).view(BF).view(256, 256)
    finite = torch.isfinite(Z)
    dY = torch.ones_like(Z)
    dZ, _ = lynx.lynx_act_backward(dY, Z, want_bias=False)
    oracle.check(torch.where(finite, dZ, 0), tuple(torch.where(finite, t, 0.0) for t in oracle.act_backward(
        dY, torch.where(finite, Z, 0))["dZ"]), "dZ")
    assert torch.isnan(dZ[torch.isnan(Z)]).all()


def test_act_gradient_against_differences():
    Z, dY = normal((4, 64), 1, 2.0), normal((4, 64), 2)
    dZ, _ = lynx.lynx_act_backward(dY, Z)
    z, h = Z.double(), 2.0 ** -20
    slope = (oracle.gelu(z + h) - oracle.gelu(z - h)) / (2 * h) * dY.double()
    assert torch.all((dZ.double() - slope).abs() <= oracle.BF16 * slope.abs() + 2.0 ** -18 * dY.double().abs())


@pytest.mark.slow
def test_act_offsets_past_32_bits():
    M, N = 2 ** 18 + 3, 8192
    dY = torch.zeros((M, N), dtype=BF, device="cuda")
    Z = torch.zeros((M, N), dtype=BF, device="cuda")
    dY[-50:], Z[-50:] = normal((50, N), 1), normal((50, N), 2)
    dZ, db = lynx.lynx_act_backward(dY, Z, dZ=dY.clone())
    want = oracle.act_backward(dY[-50:], Z[-50:])
    oracle.check(dZ[-50:], want["dZ"], "dZ")
    oracle.check(db, want["dbias"], "dbias")
    assert torch.all(dZ[:1000] == 0)


@pytest.mark.slow
def test_residual_offsets_past_32_bits():
    M, N, K = 2 ** 18 + 130, 8192, 64
    X, W, bias, _, _ = layer(M, N, K, 0, seed=5)
    R = torch.zeros((M, N), dtype=BF, device="cuda")
    R[-200:] = normal((200, N), 1)
    R[:200] = normal((200, N), 2)
    Y, _ = lynx.lynx_linear_residual(X, W, bias, R=R, skip_sparsify=True)
    for rows in (slice(0, 200), slice(M - 200, M)):
        oracle.check(Y[rows], oracle.linear_residual(X[rows], W, bias, None, None, R[rows], True, False)["Y"], "Y")


@pytest.mark.parametrize("M,N,K", [(300, 512, 576), (600, 4096, 512)])  # the 1-CTA kernel and the CTA pairs
def test_a_stalled_call_gives_up_and_the_next_one_works(M, N, K):
    X, W, bias, A, B = layer(M, N, K, 16, seed=6)
    R = normal((M, N), 9)
    want, wz = lynx.lynx_linear_residual(X, W, bias, A, B, R=R, want_Z=True)
    assert lynx.lynx_check_error() == (lynx.LYNX_OK, 0)
    lynx.lynx_debug_set_stall(True)
    try:
        lynx.lynx_linear_residual(X, W, bias, A, B, R=R, want_Z=True)
        status, code = lynx.lynx_check_error()
    finally:
        lynx.lynx_debug_set_stall(False)
    assert status == lynx.LYNX_ERR_DEVICE_TIMEOUT and code != 0
    Y, Z = lynx.lynx_linear_residual(X, W, bias, A, B, R=R, want_Z=True)
    assert lynx.lynx_check_error() == (lynx.LYNX_OK, 0)
    assert torch.equal(Y, want) and torch.equal(Z, wz)


def test_either_gemm_kernel_gives_the_same_bits():
    """Rows of a problem that the CTA pairs take, alone, where the 1-CTA kernel takes them with tiles of 32 to 128
    columns.  Dense and without an adapter nothing but the GEMM is in between: equal bits."""
    M, N, K = 2304, 2048, 512
    X, W, bias, _, _ = layer(M, N, K, 0, seed=7)
    R = normal((M, N), 9)
    for act in (NONE, GELU):
        Y, Z = lynx.lynx_linear_residual(X, W, bias, R=R, skip_sparsify=True, act=act, want_Z=True)
        for r0, r1 in ((0, 1), (0, 128), (256, 512), (1000, 1900)):
            y, z = lynx.lynx_linear_residual(X[r0:r1], W, bias, R=R[r0:r1], skip_sparsify=True, act=act, want_Z=True)
            assert torch.equal(y, Y[r0:r1]) and torch.equal(z, Z[r0:r1])


def test_few_rows_are_alone_in_their_tile():
    """The rows of a tile that are not there hold what the launch before left in shared memory: NaN here.
    The rows that are there give the bits they give among 128."""
    M, N, K, r = 128, 1000, 640, 48
    X, W, bias, _, B = layer(M, N, K, r, seed=9)
    R, T = normal((M, N), 10), normal((M, r), 11)
    vals, meta, _ = lynx.lynx_sparsify(X)
    nan = torch.full_like(X, float("nan"))
    nan_t = torch.full_like(T, float("nan"))

    def poison():
        lynx.lynx_linear(nan, W, skip_sparsify=True)
        lynx.lynx_sparse_gemm(torch.full_like(vals, float("nan")), meta, W, T=nan_t, B=B)

    dense, Z = lynx.lynx_linear_residual(X, W, bias, R=R, skip_sparsify=True, act=GELU, want_Z=True)
    sparse = lynx.lynx_sparse_gemm(vals, meta, W, bias, T=T, B=B)
    assert torch.isfinite(sparse.float()).all()
    for m in (1, 7, 8, 9, 64, 100, 127):
        poison()
        y, z = lynx.lynx_linear_residual(X[:m], W, bias, R=R[:m], skip_sparsify=True, act=GELU, want_Z=True)
        assert torch.equal(y, dense[:m]) and torch.equal(z, Z[:m]), m
        poison()
        assert torch.equal(lynx.lynx_sparse_gemm(vals[:m], meta, W, bias, T=T[:m], B=B), sparse[:m]), m
    assert lynx.lynx_check_error() == (lynx.LYNX_OK, 0)


def test_two_host_threads_on_two_streams():
    """Both at once, each on its own stream with its own buffers: what each gives alone."""
    import threading

    X, W, bias, A, B = layer(700, 1024, 512, 16, seed=8)
    R, dY = normal((700, 1024), 9), normal((700, 1024), 10)
    w = normal((1024,), 11)

    def step():
        Y, Z = lynx.lynx_linear_residual(X, W, bias, A, B, R=R, act=GELU, want_Z=True)
        N, mean, rstd = lynx.lynx_layer_norm(Y, w, want_stats=True)
        dZ, db = lynx.lynx_act_backward(dY, Z)
        return (Y, Z, N, dZ, db, *lynx.lynx_layer_norm_backward(dZ, Y, mean, rstd, w, dR=dY))

    want = step()
    torch.cuda.synchronize()
    bad = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = step()
            torch.cuda.current_stream().synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want)):
                bad.append("different")
            if lynx.lynx_check_error()[0] != lynx.LYNX_OK:
                bad.append("error")

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
