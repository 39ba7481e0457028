"""The weight in 4 bits and the layer for a few tokens, against 64 bits
(tests/adapter_oracle.py holds the formulas and derives the tolerances)."""
import pytest
import torch

from activation_sparse_gemm_lynx_b200 import lynx

import adapter_oracle as ao

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "these tests need a GPU"
    torch.cuda.set_device(0)
    lynx.library()
    yield
    torch.cuda.synchronize()


def normal(seed, *shape, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * std).bfloat16()


def guarded(shape, dtype, fill=0x5A):
    """A tensor in the middle of a buffer whose ends are checked with intact()."""
    n = int(torch.tensor(shape).prod()) * torch.empty((), dtype=dtype).element_size()
    pad = 4096
    raw = torch.full((n + 2 * pad,), fill, dtype=torch.uint8, device=DEV)
    return raw, raw[pad:pad + n].view(dtype).view(shape)


def intact(raw, t, fill=0x5A):
    n = t.numel() * t.element_size()
    return bool((raw[:4096] == fill).all()) and bool((raw[4096 + n:] == fill).all())


@pytest.mark.parametrize("zp", [False, True])
@pytest.mark.parametrize("N,K,group", [(8, 64, 32), (8, 64, 64), (40, 128, 128), (1000, 576, 64), (264, 1088, 32),
                                       (136, 4224, 128)])
def test_quantize_and_back_are_exact(N, K, group, zp):
    W = normal(N + K, N, K, std=0.05)
    W[1, :group] = 0                     # a group of zeros
    W[2, :group] = W[2, :group].abs()    # one sign only
    W[3, :group] = -W[3, :group].abs()
    W[4, 0] = 30.0                       # an outlier
    W[5] = W[5] * 2.0 ** -120            # near the end of the range
    W[6, :group] = 2.0 ** -133           # smallest magnitude: the scale rounds to 0
    raws = [guarded(s, d) for s, d in (((N, K // 2), torch.uint8), ((K // group, N), torch.bfloat16),
                                       ((K // group, N), torch.uint8), ((N, K), torch.bfloat16))]
    (r0, Wq), (r1, sc), (r2, ze), (r3, back) = raws
    lynx.lynx_w4_quantize(W, group, zp, Wq=Wq, scales=sc, zeros=ze if zp else None)
    lynx.lynx_w4_dequantize(Wq, sc, ze if zp else None, W=back)
    q, s, z = ao.w4_quantize(W, group, zp)
    assert torch.equal(sc.double(), s.t())
    if zp:
        assert torch.equal(ze.double(), z.t())
    assert torch.equal(Wq, ao.w4_pack(q))
    assert torch.equal(back, ao.w4_values(q, s, z).bfloat16())
    assert all(intact(r, t) for r, t in raws)


def w4_case(seed, N, K, group, zp):
    """Random nibbles, scales and zero points: all 16 values, whatever a quantiser would do."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randint(0, 16, (N, K), generator=g, device=DEV)
    s = (torch.rand(N, K // group, generator=g, device=DEV) * 0.02 + 1e-3).bfloat16()
    z = torch.randint(0, 16, (N, K // group), generator=g, device=DEV)
    Wq, sc = ao.w4_pack(q), s.t().contiguous()
    ze = z.to(torch.uint8).t().contiguous() if zp else None
    zd = z.double() if zp else torch.full_like(s, 8.0, dtype=torch.float64)
    return Wq, sc, ze, ao.w4_values(q.double(), s.double(), zd)


CASES = [(1, 8, 64, 32, 0, False), (1, 8, 64, 64, 16, True), (2, 24, 128, 128, 64, False), (7, 136, 192, 32, 0, True),
         (8, 520, 576, 64, 16, False), (9, 520, 576, 32, 144, False), (15, 264, 640, 128, 64, True),
         (16, 1000, 1088, 64, 256, False), (17, 1000, 1088, 32, 0, False), (24, 128, 4224, 128, 64, False),
         (31, 72, 4160, 64, 48, True), (32, 4104, 512, 128, 64, False), (1, 4104, 4096, 128, 64, True),
         (1, 128, 12288, 32, 0, False), (5, 12296, 256, 64, 16, False), (3, 16, 16384, 128, 256, False)]


@pytest.mark.parametrize("zp", [False, True])
@pytest.mark.parametrize("M,N,K,group,r,act", CASES)
def test_linear_w4(M, N, K, group, r, act, zp):
    Wq, sc, ze, W = w4_case(M * N + K, N, K, group, zp)
    X, bias = normal(1, M, K), normal(2, N)
    A, B = (normal(3, r, K, std=0.02), normal(4, N, r, std=0.2)) if r else (None, None)
    raw, Y = guarded((M, N), torch.bfloat16)
    need = lynx.lynx_linear_w4_workspace_bytes(M, N, K, r)
    wraw, ws = guarded((max(need, 1),), torch.uint8)
    lynx.lynx_linear_w4(X, Wq, sc, ze, bias, A, B, act=int(act), Y=Y, workspace=ws if r else None)
    ref, tol = ao.linear_w4(X, W, bias, A, B, act)
    off = (Y.double() - ref).abs() / tol
    assert float(off.max()) <= 1, float(off.max())
    assert intact(raw, Y) and intact(wraw, ws)
    # again, without bias, into a buffer of its own; and the same call gives the same bits
    Y2 = lynx.lynx_linear_w4(X, Wq, sc, ze, None, A, B)
    ref, tol = ao.linear_w4(X, W, None, A, B)
    assert bool(((Y2.double() - ref).abs() <= tol).all())
    assert torch.equal(Y2, lynx.lynx_linear_w4(X, Wq, sc, ze, None, A, B))


def test_rows_do_not_touch_each_other():
    """An infinity or a NaN in one token stays in its row."""
    Wq, sc, ze, W = w4_case(9, 264, 640, 64, True)
    A, B = normal(3, 32, 640, std=0.02), normal(4, 264, 32, std=0.2)
    X = normal(1, 6, 640)
    Y = lynx.lynx_linear_w4(X, Wq, sc, ze, None, A, B)
    X2 = X.clone()
    X2[2, 5], X2[4, 639] = float("inf"), float("nan")
    Y2 = lynx.lynx_linear_w4(X2, Wq, sc, ze, None, A, B)
    rest = [0, 1, 3, 5]
    assert torch.equal(Y[rest], Y2[rest])
    assert not bool(torch.isfinite(Y2[[2, 4]]).any())


def test_two_streams_at_once():
    """Two calls that overlap, each with its own buffers on its own stream."""
    Wq, sc, ze, W = w4_case(10, 4096, 2048, 128, False)
    A, B = normal(3, 64, 2048, std=0.02), normal(4, 4096, 64, std=0.2)
    Xs = [normal(20 + i, m, 2048) for i, m in enumerate((1, 32))]
    want = [lynx.lynx_linear_w4(x, Wq, sc, ze, None, A, B) for x in Xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(lynx.lynx_linear_w4(Xs[i], Wq, sc, ze, None, A, B, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in (0, 1) for y in got[i])


def test_graph_replay_with_new_inputs():
    Wq, sc, ze, W = w4_case(11, 1032, 1024, 64, True)
    A, B = normal(3, 64, 1024, std=0.02), normal(4, 1032, 64, std=0.2)
    X = normal(1, 3, 1024)
    lynx.lynx_linear_w4(X, Wq, sc, ze, None, A, B)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Y = lynx.lynx_linear_w4(X, Wq, sc, ze, None, A, B)
        Y2 = lynx.lynx_linear_w4(X, Wq, sc, ze, None, A, B, act=lynx.LYNX_ACT_GELU_TANH)
    for seed in (50, 51):
        X.copy_(normal(seed, 3, 1024))
        g.replay()
        torch.cuda.synchronize()
        for y, act in ((Y, False), (Y2, True)):
            ref, tol = ao.linear_w4(X, W, None, A, B, act)
            assert bool(((y.double() - ref).abs() <= tol).all())


def test_dequantized_weight_serves_the_sparse_layer():
    """The 4-bit weight's way to many tokens: dequantise, then lynx_linear_dense."""
    W = normal(30, 512, 576, std=0.05)
    Wq, sc, ze = lynx.lynx_w4_quantize(W, 64, True)
    X = normal(31, 32, 576)
    many = lynx.lynx_linear_dense(X, lynx.lynx_w4_dequantize(Wq, sc, ze))
    few = lynx.lynx_linear_w4(X, Wq, sc, ze)
    q, s, z = ao.w4_quantize(W, 64, True)
    v = ao.w4_values(q, s, z)
    ref, tol = ao.linear_w4(X, v)
    assert bool(((few.double() - ref).abs() <= tol).all())
    # the dense layer sees each weight rounded to bf16 once
    assert bool(((many.double() - ref).abs() <= tol + ao.BF * (X.double().abs() @ v.abs().t())).all())


def test_bindings_refuse():
    Wq, sc, ze, _ = w4_case(12, 64, 256, 64, True)
    X = normal(1, 4, 256)
    with pytest.raises(lynx.LynxError):
        lynx.lynx_linear_w4(normal(1, 33, 256), Wq, sc)
    with pytest.raises(ValueError):
        lynx.lynx_linear_w4(X[:, :128], Wq, sc)
    with pytest.raises(ValueError):
        lynx.lynx_linear_w4(X, Wq, sc.t().contiguous())
    with pytest.raises(TypeError):
        lynx.lynx_linear_w4(X.float(), Wq, sc)
    with pytest.raises(ValueError):
        lynx.lynx_linear_w4(X, Wq, sc, ze[:2])
    with pytest.raises(ValueError):
        lynx.lynx_linear_w4(X, Wq, sc, A=normal(1, 16, 256))
    with pytest.raises(lynx.LynxError):
        lynx.lynx_linear_w4(X, Wq, sc, A=normal(1, 24, 256), B=normal(1, 64, 24))
    with pytest.raises(lynx.LynxError):
        lynx.lynx_w4_quantize(normal(1, 64, 192), 128)
    with pytest.raises(lynx.LynxError):
        lynx.lynx_linear_w4(X, Wq, sc, act=7)


def test_arguments_of_other_kinds_are_refused():
    Wq, sc, ze, _ = w4_case(12, 64, 256, 64, True)
    X, W = normal(1, 4, 256), normal(2, 64, 256)
    for act in (1 << 32, 0.0, None, "gelu"):  # the first is 0 in 32 bits
        with pytest.raises(TypeError):
            lynx.lynx_linear_w4(X, Wq, sc, act=act)
    for group in ((1 << 32) + 64, 64.0, None):
        with pytest.raises(TypeError):
            lynx.lynx_w4_quantize(W, group)
    with pytest.raises(TypeError):
        lynx.lynx_w4_quantize(W, 64, zero_points=torch.zeros(2))
    with pytest.raises(TypeError):
        lynx.lynx_linear_w4(X, Wq, sc, stream=0)
    with pytest.raises(TypeError):
        lynx.lynx_linear_w4([1.0], Wq, sc)
    with pytest.raises(ValueError):
        lynx.lynx_linear_w4(None, Wq, sc)
    with pytest.raises(lynx.LynxError):
        lynx.lynx_linear_w4(X, Wq, sc, ze, Y=X[:, :64].contiguous(), workspace=None, A=normal(3, 16, 256),
                            B=normal(4, 64, 16)[:, :16], act=2)
    Y = torch.empty(4, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(lynx.LynxError):  # the output in the place of the bias
        lynx.lynx_linear_w4(X, Wq, sc, ze, Y[0], Y=Y)
