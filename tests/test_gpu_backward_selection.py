"""dX is the gradient of the layer that ran: the selection is the forward pass's
metadata, the values are the checkpoint's."""
import math

import pytest
import torch

from activation_sparse_gemm_lynx_b200 import lynx

import adapter_oracle as ao
import selection_oracle as so
from norms import rounded_once
from test_gpu_w4 import DEV, guarded, intact, normal

pytestmark = pytest.mark.gpu
FORMATS = [lynx.LYNX_CKPT8_INT8, lynx.LYNX_CKPT8_E4M3]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    torch.cuda.set_device(0)
    lynx.library()
    yield
    st, code = lynx.lynx_check_error()
    assert st == lynx.LYNX_OK, (st, code)


def activations(seed, M, K, kind):
    z = normal(seed, M, K).float()
    if kind == "gelu":
        z = z - 0.5
        return (0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))).bfloat16()
    return torch.where(normal(seed + 1, M, K).float() < -1.4, z, z * 0.05).bfloat16()


def checkpoint(X, fmt):
    q, e = lynx.lynx_ckpt8_store(X, fmt)
    return q, e, ao.ckpt8_values(q.float().double(), e.long(), fmt == lynx.LYNX_CKPT8_INT8)


@pytest.mark.parametrize("fmt,most", [(lynx.LYNX_CKPT8_INT8, 0.02), (lynx.LYNX_CKPT8_E4M3, 0.005)])
@pytest.mark.parametrize("kind", ["mixture", "gelu"])
@pytest.mark.parametrize("M,N,K,r", [(300, 576, 4096, 64), (100, 192, 1088, 0), (1, 64, 12288, 16)])
def test_the_gradient_of_the_layer_that_ran(M, N, K, r, kind, fmt, most):
    """lynx_linear, then dX, against the 64-bit derivative at the X of the forward pass.

    What 8 bits for x cost is |formula at the checkpoint - derivative at X|, in 64 bits; the
    kernel adds its rounding to that and nothing else (triangle inequality).  The header
    names that cost at K = 4096: 0.02 (int8) and 0.005 (e4m3) of the norm.  Most of it is
    the signs of values stored as 0, whose share D / Lk of dX each entry loses; with D the
    sum of K random terms and Lk that of K magnitudes it falls as 1 / sqrt(K), so shorter
    rows pay more and the figure is asserted where it is stated."""
    X, W = activations(1, M, K, kind), normal(3, N, K, std=0.04)
    A, B = (normal(4, r, K, std=0.05), normal(5, N, r, std=0.05)) if r else (None, None)
    ws = torch.empty(lynx.lynx_workspace_bytes(M, N, K, r or 64), dtype=torch.uint8, device=DEV)
    lynx.lynx_linear(X, W, None, A, B, workspace=ws)
    meta = lynx.lynx_workspace_meta(ws, M, K).clone()
    q, e = lynx.lynx_ckpt8_store(X, fmt)
    G = normal(6, M, K, std=1e-3)
    dT = normal(7, M, r, std=1e-3) if r else None
    dX = lynx.lynx_sparsify_backward(G, q, e, dT, A, meta=meta)
    true, _ = ao.sparsify_backward(G, X.double(), dT, A)
    x = ao.ckpt8_values(q.float().double(), e.long(), fmt == lynx.LYNX_CKPT8_INT8)
    formula, _ = so.gradient(G, x, so.from_metadata(meta, M, K), dT, A)
    cost = float((formula - true).norm())
    rounding = 1.1 * float((formula.bfloat16().double() - formula).norm()) + 2.0 ** -12 * float(formula.norm())
    assert float((dX.double() - true).norm()) <= cost + rounding
    if K == 4096:
        assert float((dX.double() - true).norm() / true.norm()) <= most
    # and the call without the metadata is what the header says it is
    if r == 64:
        assert float((lynx.lynx_sparsify_backward(G, q, e, dT, A).double() - true).norm() / true.norm()) > 0.1


@pytest.mark.parametrize("M,K", [(1, 64), (257, 1088), (300, 4096), (128, 192)])
def test_the_workspace_holds_the_selection(M, K):
    X = activations(2, M, K, "mixture")
    W = normal(3, 264, K)
    keep = ao.keep(X.double())
    assert torch.equal(so.from_metadata(lynx.lynx_sparsify(X)[1], M, K), keep)
    A, B = normal(4, 32, K), normal(5, 264, 32)
    for a, b in ((None, None), (A, B)):
        ws = torch.empty(lynx.lynx_workspace_bytes(M, 264, K, 32 if a is not None else 64), dtype=torch.uint8, device=DEV)
        lynx.lynx_linear_act(X, W, None, a, b, workspace=ws)
        # (columns past K of the last block, K % 128 = 64, belong to nobody)
        assert torch.equal(so.from_metadata(lynx.lynx_workspace_meta(ws, M, K), M, K), keep)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K,r", [(1, 64, 0), (1, 64, 16), (2, 128, 64), (15, 192, 32), (16, 576, 48), (17, 1088, 0),
                                   (257, 1088, 64), (300, 4160, 16), (33, 12288, 64), (5, 16448, 256), (64, 2048, 144),
                                   (3, 65536, 16), (1031, 256, 128), (129, 320, 0), (600, 12288, 64)])
def test_against_the_formula(M, K, r, fmt):
    X = activations(M + K, M, K, "mixture")
    X[0, :32] = 0
    X[-1] = 0 if M > 1 else X[-1]
    X[M // 2, 32:36] = 1.0
    _, meta, _ = lynx.lynx_sparsify(X)
    m = so.from_metadata(meta, M, K)
    q, e, x = checkpoint(X, fmt)
    G = normal(2, M, K)
    dT, A = (normal(3, M, r), normal(4, r, K, std=0.2)) if r else (None, None)
    raws = [guarded((M, K), torch.bfloat16), guarded((lynx.lynx_sparsify_backward_workspace_bytes(M, K),), torch.uint8)]
    (_, dX), (_, ws) = raws
    lynx.lynx_sparsify_backward(G, q, e, dT, A, dX, ws, meta=meta)
    ref, tol = so.gradient(G, x, m, dT, A)
    assert bool(((dX.double() - ref).abs() <= tol).all())
    if M * K >= 500:
        rounded_once(dX, ref)
    assert all(intact(r_, t) for r_, t in raws)
    ws.fill_(0xFF)
    assert torch.equal(dX, lynx.lynx_sparsify_backward(G, q, e, dT, A, workspace=ws, meta=meta))


@pytest.mark.parametrize("fmt", FORMATS)
def test_any_metadata(fmt):
    """Every nibble, the ones no selection makes among them (one position twice keeps one
    value), and rows whose kept values are all zero."""
    M, K = 300, 1088
    g = torch.Generator(device=DEV).manual_seed(1)
    meta = torch.randint(0, 256, (lynx.lynx_meta_bytes(M, K),), generator=g, device=DEV, dtype=torch.uint8)
    m = so.from_metadata(meta, M, K)
    X = normal(2, M, K)
    X[5] = torch.where(m[5] > 0, 0.0, X[5].double()).bfloat16()
    q, e, x = checkpoint(X, fmt)
    G = normal(3, M, K)
    dX = lynx.lynx_sparsify_backward(G, q, e, meta=meta)
    ref, tol = so.gradient(G, x, m)
    assert bool(((dX.double() - ref).abs() <= tol).all())
    assert torch.equal(dX[5], torch.where(m[5] > 0, G[5].double(), 0.0).bfloat16())
    # what is dropped is not read
    for bad in (float("inf"), float("nan"), torch.finfo(torch.bfloat16).min):
        assert torch.equal(lynx.lynx_sparsify_backward(torch.where(m > 0, G, bad), q, e, meta=meta), dX)


def test_against_differences():
    """Central differences of sum(G * S(x)) with the selection fixed, in 64 bits."""
    M, K, h = 3, 128, 2.0 ** -20
    X = activations(8, M, K, "mixture")
    _, meta, _ = lynx.lynx_sparsify(X)
    m = so.from_metadata(meta, M, K)
    q, e, x = checkpoint(X, lynx.LYNX_CKPT8_INT8)
    G = normal(9, M, K)
    dX = lynx.lynx_sparsify_backward(G, q, e, meta=meta).double()
    _, tol = so.gradient(G, x, m)
    steps = torch.eye(K, dtype=torch.float64, device=DEV) * h
    for i in range(M):
        mi = m[i].expand(K, K)
        num = ((so.layer(x[i] + steps, mi) - so.layer(x[i] - steps, mi)) @ G[i].double()) / (2 * h)
        smooth = x[i].abs() > 4 * h  # |x| has no derivative at 0
        assert float(smooth.double().mean()) > 0.5
        # the difference's own error: h^2 curvature and 64-bit cancellation, both below 1e-8
        assert bool(((num - dX[i]).abs() <= tol[i] + 1e-8)[smooth].all())


def test_graph_replay_and_streams():
    M, N, K, r = 300, 520, 640, 64
    X, W = activations(1, M, K, "gelu"), normal(2, N, K, std=0.04)
    A, B, G, dT = normal(3, r, K), normal(4, N, r), normal(5, M, K), normal(6, M, r)
    ws = torch.empty(lynx.lynx_workspace_bytes(M, N, K, r), dtype=torch.uint8, device=DEV)

    def step():
        lynx.lynx_linear(X, W, None, A, B, workspace=ws)
        q, e = lynx.lynx_ckpt8_store(X)
        return lynx.lynx_sparsify_backward(G, q, e, dT, A, meta=lynx.lynx_workspace_meta(ws, M, K))

    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    q, e = lynx.lynx_ckpt8_store(X)
    meta = lynx.lynx_workspace_meta(ws, M, K).clone()
    s.wait_stream(torch.cuda.current_stream())
    got = [lynx.lynx_sparsify_backward(G, q, e, dT, A, stream=s, meta=meta) for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    X.copy_(activations(20, M, K, "mixture"))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, step()) and not torch.equal(out, want)


def test_bindings_refuse():
    M, K = 8, 128
    X, G = normal(1, M, K), normal(2, M, K)
    _, meta, _ = lynx.lynx_sparsify(X)
    q, e = lynx.lynx_ckpt8_store(X)
    with pytest.raises(ValueError):
        lynx.lynx_sparsify_backward(G, q, e, meta=meta[:-1])
    with pytest.raises(TypeError):
        lynx.lynx_sparsify_backward(G, q, e, meta=meta.view(torch.int32))
    with pytest.raises(ValueError):
        lynx.lynx_sparsify_backward(G, q, e, meta=meta.cpu())
    with pytest.raises(ValueError):
        lynx.lynx_sparsify_backward(G, q, e, meta=torch.cat([meta, meta])[::2])
    with pytest.raises(lynx.LynxError):  # the output in the place of the metadata
        lynx.lynx_sparsify_backward(G, q, e, meta=meta, dX=meta[:2 * M * K].view(torch.bfloat16).view(M, K))
    with pytest.raises(lynx.LynxError):  # not on 16 bytes
        lynx.lynx_sparsify_backward(G, q, e, meta=torch.cat([meta, meta])[8:])
    with pytest.raises(ValueError):
        lynx.lynx_workspace_meta(torch.empty(100, dtype=torch.uint8, device=DEV), M, K)
