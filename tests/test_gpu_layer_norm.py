"""lynx_layer_norm and lynx_layer_norm_backward against the formulas in 64 bits."""
import pytest
import torch

import block_oracle as oracle
from activation_sparse_gemm_lynx_b200 import lynx

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
EPS = 1e-6

# one piece, odd pieces, the widths where the threads of a row, the rows of a block or the ring's
# depth change, the framework's widths and the widest
SHAPES = [(1, 8), (3, 64), (1, 4096), (300, 1088), (257, 576), (33, 1000), (1024, 1024), (64, 1032), (5, 2056), (700, 4096),
          (150, 4104), (9, 8192), (9, 8200), (40, 12288), (3, 16392), (2, 32768)]


def stream(M, K, seed, offset=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn((M, K), generator=g, device="cuda") * (0.5 + torch.rand((M, 1), generator=g, device="cuda"))
    return (z + offset + 0.2 * torch.randn((M, 1), generator=g, device="cuda")).to(BF)


def vector(K, seed, mean, std):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (mean + std * torch.randn(K, generator=g, device="cuda")).to(BF)


def gradient(M, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((M, K), generator=g, device="cuda").to(BF)


@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("M,K", SHAPES)
def test_forward(M, K, affine):
    X = stream(M, K, M + K)
    w, b = (vector(K, 1, 1.0, 0.2), vector(K, 2, 0.0, 0.1)) if affine else (None, None)
    Y, mean, rstd = lynx.lynx_layer_norm(X, w, b, eps=EPS, want_stats=True)
    want = oracle.layer_norm(X, w, b, EPS)
    oracle.check(Y, want["Y"], "Y")
    oracle.check(mean, want["mean"], "mean")
    oracle.check(rstd, want["rstd"], "rstd")
    # without the statistics the rows are the same, bit for bit
    assert torch.equal(lynx.lynx_layer_norm(X, w, b, eps=EPS), Y)


@pytest.mark.parametrize("which", ["weight", "bias"])
def test_forward_with_one_of_the_two(which):
    X = stream(20, 1088, 5)
    w = vector(1088, 1, 1.0, 0.2) if which == "weight" else None
    b = vector(1088, 2, 0.0, 0.1) if which == "bias" else None
    oracle.check(lynx.lynx_layer_norm(X, w, b, eps=EPS), oracle.layer_norm(X, w, b, EPS)["Y"], "Y")


def test_rows_far_from_zero_keep_their_variance():
    X = stream(64, 4096, 3, offset=200.0)  # x - mean is about 1 % of x
    Y, mean, rstd = lynx.lynx_layer_norm(X, eps=EPS, want_stats=True)
    want = oracle.layer_norm(X, None, None, EPS)
    oracle.check(Y, want["Y"], "Y")
    oracle.check(rstd, want["rstd"], "rstd")


def test_constant_rows_large_and_small_rows():
    X = stream(6, 1024, 4)
    X[0] = 3.0
    X[1] = 0.0
    X[2] = stream(1, 1024, 5)[0] * 2.0 ** 55
    X[3] = stream(1, 1024, 6)[0] * 2.0 ** -60
    Y, mean, rstd = lynx.lynx_layer_norm(X, eps=EPS, want_stats=True)
    want = oracle.layer_norm(X, None, None, EPS)
    oracle.check(Y, want["Y"], "Y")
    assert torch.all(Y[:2] == 0)
    assert float(mean[0]) == 3.0 and float(mean[1]) == 0.0
    assert torch.allclose(rstd[:2], torch.full((2,), 1e3, device="cuda"), rtol=1e-5)


def test_a_row_that_is_not_finite_stays_alone():
    X = stream(40, 576, 7)
    X[3, 100] = float("inf")
    X[17, 575] = float("nan")
    Y, mean, rstd = lynx.lynx_layer_norm(X, eps=EPS, want_stats=True)
    rows = [i for i in range(40) if i not in (3, 17)]
    want = oracle.layer_norm(X[rows], None, None, EPS)
    oracle.check(Y[rows], want["Y"], "Y")
    assert torch.isnan(Y[3]).all() and torch.isnan(Y[17]).all()
    dY = gradient(40, 576, 8)
    dX, _, _ = lynx.lynx_layer_norm_backward(dY, X, mean, rstd)
    assert torch.isnan(dX[[3, 17]]).all()
    oracle.check(dX[rows], oracle.layer_norm_backward(dY[rows], X[rows], mean[rows], rstd[rows], None, None)["dX"], "dX")


@pytest.mark.parametrize("affine,branch", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("M,K", SHAPES)
def test_backward(M, K, affine, branch):
    X, dY = stream(M, K, M + K), gradient(M, K, 1)
    w = vector(K, 1, 1.0, 0.2) if affine else None
    dR = gradient(M, K, 2) if branch else None
    _, mean, rstd = lynx.lynx_layer_norm(X, w, None, eps=EPS, want_stats=True)
    dX, dw, db = lynx.lynx_layer_norm_backward(dY, X, mean, rstd, w, dR=dR)
    want = oracle.layer_norm_backward(dY, X, mean, rstd, w, dR)
    oracle.check(dX, want["dX"], "dX")
    oracle.check(dw, want["dweight"], "dweight")
    oracle.check(db, want["dbias"], "dbias")


@pytest.mark.parametrize("K", [576, 4096, 12288])
def test_backward_with_only_what_is_wanted(K):
    M = 70
    X, dY, w = stream(M, K, 1), gradient(M, K, 1), vector(K, 1, 1.0, 0.2)
    _, mean, rstd = lynx.lynx_layer_norm(X, w, None, eps=EPS, want_stats=True)
    dX, dw, db = lynx.lynx_layer_norm_backward(dY, X, mean, rstd, w)
    a, none, b = lynx.lynx_layer_norm_backward(dY, X, mean, rstd, w, want_weight=False)
    assert none is None and torch.equal(b, db) and torch.equal(a, dX)
    a, c, none = lynx.lynx_layer_norm_backward(dY, X, mean, rstd, w, want_bias=False)
    assert none is None and torch.equal(c, dw) and torch.equal(a, dX)
    a, n1, n2 = lynx.lynx_layer_norm_backward(dY, X, mean, rstd, w, want_weight=False, want_bias=False)
    assert n1 is None and n2 is None and torch.equal(a, dX)


@pytest.mark.parametrize("M,K", [(300, 1088), (700, 4096), (40, 12288)])
def test_equal_calls_give_equal_bits_and_dr_may_be_dx(M, K):
    X, dY, w, dR = stream(M, K, 1), gradient(M, K, 1), vector(K, 1, 1.0, 0.2), gradient(M, K, 2)
    _, mean, rstd = lynx.lynx_layer_norm(X, w, None, eps=EPS, want_stats=True)
    first = lynx.lynx_layer_norm_backward(dY, X, mean, rstd, w, dR=dR)
    here = dR.clone()
    second = lynx.lynx_layer_norm_backward(dY, X, mean, rstd, w, dR=here, dX=here)
    assert second[0] is here or second[0].data_ptr() == here.data_ptr()
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_gradients_against_differences():
    """dL/d(everything) for L = sum(Y c) by central differences of the formula in 64 bits."""
    M, K = 4, 64
    X, w, b, c = stream(M, K, 1), vector(K, 1, 1.0, 0.2), vector(K, 2, 0.0, 0.1), gradient(M, K, 3)
    _, mean, rstd = lynx.lynx_layer_norm(X, w, b, eps=1e-3, want_stats=True)
    dX, dw, db = lynx.lynx_layer_norm_backward(c, X, mean, rstd, w)

    def loss(x, ww, bb):
        d = x - x.mean(1, keepdim=True)
        return ((d * ((d * d).mean(1, keepdim=True) + 1e-3) ** -0.5 * ww + bb) * c.double()).sum()

    at = [X.double(), w.double(), b.double()]
    h = 2.0 ** -18
    for i, got in enumerate((dX, dw, db)):
        for j in range(0, at[i].numel(), 7):
            up, down = [t.clone() for t in at], [t.clone() for t in at]
            up[i].view(-1)[j] += h
            down[i].view(-1)[j] -= h
            slope = float((loss(*up) - loss(*down)) / (2 * h))
            # differences are off by h^2 and 2^-52 |L| / h, both far below bf16's half step of a gradient of order 1
            assert abs(float(got.double().view(-1)[j]) - slope) <= oracle.BF16 * abs(slope) + 1e-4


def test_nothing_behind_the_last_row_is_written():
    M, K = 37, 1000
    room = torch.full((M + 3, K), 7.0, dtype=BF, device="cuda")
    stats = torch.full((2, 64), 7.0, device="cuda")
    X = stream(M, K, 1)
    lynx.lynx_layer_norm(X, eps=EPS, want_stats=True, Y=room[:M], mean=stats[0, :M], rstd=stats[1, :M])
    assert torch.all(room[M:] == 7.0) and torch.all(stats[:, M:] == 7.0)
    grads = torch.full((M + 3, K), 7.0, dtype=BF, device="cuda")
    need = lynx.lynx_layer_norm_backward_workspace_bytes(M, K)
    ws = torch.full((need + 256,), 5, dtype=torch.uint8, device="cuda")
    lynx.lynx_layer_norm_backward(gradient(M, K, 1), X, stats[0, :M], stats[1, :M], dX=grads[:M], workspace=ws)
    assert torch.all(grads[M:] == 7.0) and torch.all(ws[need:] == 5)


def test_another_stream_and_a_captured_graph():
    M, K = 300, 4096
    X, dY, w = stream(M, K, 1), gradient(M, K, 1), vector(K, 1, 1.0, 0.2)
    Y, mean, rstd = lynx.lynx_layer_norm(X, w, eps=EPS, want_stats=True)
    want = (Y,) + lynx.lynx_layer_norm_backward(dY, X, mean, rstd, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Y2, m2, r2 = lynx.lynx_layer_norm(X, w, eps=EPS, want_stats=True, stream=side)
    got = (Y2,) + lynx.lynx_layer_norm_backward(dY, X, m2, r2, w, stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    bufs = dict(dX=torch.empty_like(X), dweight=torch.empty_like(w), dbias=torch.empty_like(w))
    ws = torch.empty(lynx.lynx_layer_norm_backward_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    Yg, mg, rg = torch.empty_like(X), torch.empty_like(mean), torch.empty_like(rstd)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lynx.lynx_layer_norm(X, w, eps=EPS, want_stats=True, Y=Yg, mean=mg, rstd=rg)
        lynx.lynx_layer_norm_backward(dY, X, mg, rg, w, workspace=ws, **bufs)
    X2 = stream(M, K, 9)
    for source in (X2, X.clone()):  # other values through the same graph, twice
        X.copy_(source)
        graph.replay()
        graph.replay()
        Yw, mw, rw = lynx.lynx_layer_norm(X, w, eps=EPS, want_stats=True)
        torch.cuda.synchronize()
        assert torch.equal(Yg, Yw)
        for a, b in zip(bufs.values(), lynx.lynx_layer_norm_backward(dY, X, mw, rw, w)):
            assert torch.equal(a, b)


@pytest.mark.slow
def test_offsets_past_32_bits():
    M, K = 2 ** 18 + 5, 8192  # M K passes 2^31
    X = torch.zeros((M, K), dtype=BF, device="cuda")
    tail = stream(64, K, 1)
    X[-64:] = tail
    dY = torch.zeros((M, K), dtype=BF, device="cuda")
    dY[-64:] = gradient(64, K, 2)
    Y, mean, rstd = lynx.lynx_layer_norm(X, eps=EPS, want_stats=True)
    oracle.check(Y[-64:], oracle.layer_norm(tail, None, None, EPS)["Y"], "Y")
    assert torch.all(Y[:1000] == 0)
    dX, dw, db = lynx.lynx_layer_norm_backward(dY, X, mean, rstd, None, dX=Y)
    want = oracle.layer_norm_backward(dY[-64:], tail, mean[-64:], rstd[-64:], None, None)
    oracle.check(dX[-64:], want["dX"], "dX")
    oracle.check(dw, want["dweight"], "dweight")  # the other rows add exact zeros
    oracle.check(db, want["dbias"], "dbias")
