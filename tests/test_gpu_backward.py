"""The backward pass from an 8-bit checkpoint against 64 bits (formulas and
tolerances in tests/adapter_oracle.py), and a whole training step with it."""
import pytest
import torch

from activation_sparse_gemm_lynx_b200 import lynx

import adapter_oracle as ao
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


def heavy(seed, M, K):
    X = normal(seed, M, K)
    return torch.where(normal(seed + 1, M, K).float() < -1.4, X, X * 0.05)


def checkpoint(X, fmt):
    q, e = lynx.lynx_ckpt8_store(X, fmt)
    return q, e, ao.ckpt8_values(q.float().double(), e.long(), fmt == lynx.LYNX_CKPT8_INT8)


def within(got, ref, tol, what=""):
    off = (got.double() - ref).abs() / tol
    assert float(off.max()) <= 1, (what, float(off.max()), int(off.argmax()))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K,r", [(1, 8, 64, 16), (2, 16, 64, 64), (127, 136, 128, 32), (128, 128, 128, 64),
                                     (129, 264, 192, 48), (300, 1000, 576, 16), (520, 520, 1088, 144),
                                     (1, 4104, 4096, 64), (1000, 640, 256, 256), (257, 3080, 2112, 64),
                                     (2049, 72, 64, 80), (384, 1024, 1024, 128), (300, 4104, 320, 256),
                                     (1025, 2056, 128, 192), (70, 12296, 64, 240), (1500, 1032, 2048, 112)])
def test_lora_backward(M, N, K, r, fmt):
    q, e, x = checkpoint(heavy(M + K, M, K), fmt)
    dY, A, B = normal(2, M, N, std=1e-2), normal(3, r, K, std=0.1), normal(4, N, r, std=0.1)
    need = lynx.lynx_lora_backward_workspace_bytes(M, N, K, r)
    raws = [guarded((r, K), torch.bfloat16), guarded((N, r), torch.bfloat16), guarded((M, r), torch.bfloat16),
            guarded((need,), torch.uint8)]
    (_, dA), (_, dB), (_, dT), (_, ws) = raws
    lynx.lynx_lora_backward(dY, q, e, A, B, dA, dB, dT, ws)
    ref = ao.lora_backward(dY, x, A, B)
    for name, got in (("dT", dT), ("dB", dB), ("dA", dA)):
        within(got, *ref[name], name)
    assert all(intact(r_, t) for r_, t in raws)
    # equal calls give equal bits, whatever the workspace held
    ws.fill_(0xFF)
    for a, b in zip((dA, dB, dT), lynx.lynx_lora_backward(dY, q, e, A, B, workspace=ws)):
        assert torch.equal(a, b)


def test_lora_backward_without_dT(fmt=lynx.LYNX_CKPT8_INT8):
    """dT is optional in the C ABI."""
    M, N, K, r = 200, 264, 320, 32
    q, e, x = checkpoint(heavy(1, M, K), fmt)
    dY, A, B = normal(2, M, N), normal(3, r, K), normal(4, N, r)
    want = lynx.lynx_lora_backward(dY, q, e, A, B)
    dA, dB = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = torch.empty(lynx.lynx_lora_backward_workspace_bytes(M, N, K, r), dtype=torch.uint8, device=DEV)
    p = lynx._ptr
    st = lynx.library().lynx_lora_backward(p(dY), p(q), p(e), p(A), p(B), M, N, K, r, fmt, p(dA), p(dB), None,
                                           p(ws), ws.numel(), lynx._stream(None))
    assert st == lynx.LYNX_OK
    assert torch.equal(dA, want[0]) and torch.equal(dB, want[1])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K,r", [(1, 64, 0), (1, 64, 16), (2, 128, 64), (15, 192, 32), (16, 576, 48), (17, 1088, 0),
                                   (257, 1088, 64), (300, 4160, 16), (33, 12288, 64), (5, 16448, 256), (64, 2048, 144),
                                   (3, 65536, 16), (1031, 256, 128), (2, 98368, 32)])
def test_sparsify_backward(M, K, r, fmt):
    X = heavy(M + K, M, K)
    X[0, :32] = 0
    X[-1] = 0 if M > 1 else X[-1]     # a row that keeps nothing
    X[M // 2, 32:36] = 1.0            # ties
    q, e, x = checkpoint(X, fmt)
    G = normal(2, M, K)
    dT, A = (normal(3, M, r), normal(4, r, K, std=0.2)) if r else (None, None)
    raws = [guarded((M, K), torch.bfloat16), guarded((lynx.lynx_sparsify_backward_workspace_bytes(M, K),), torch.uint8)]
    (_, dX), (_, ws) = raws
    lynx.lynx_sparsify_backward(G, q, e, dT, A, dX, ws)
    within(dX, *ao.sparsify_backward(G, x, dT, A))
    assert all(intact(r_, t) for r_, t in raws)
    ws.fill_(0xFF)
    assert torch.equal(dX, lynx.lynx_sparsify_backward(G, q, e, dT, A, workspace=ws))


@pytest.mark.parametrize("fmt", FORMATS)
def test_sparsify_backward_against_differences(fmt):
    """The kernel's gradient against central differences of sum(G * S(x)) in 64
    bits.  Only entries whose group is settled (the gap between kept and dropped
    magnitudes is over the step) have one."""
    M, K, h = 3, 128, 2.0 ** -20
    q, e, x = checkpoint(normal(8, M, K), fmt)
    G = normal(9, M, K)
    dX = lynx.lynx_sparsify_backward(G, q, e).double()
    _, tol = ao.sparsify_backward(G, x)
    a = x.abs().reshape(M, -1, 4).sort(dim=2).values
    settled = (a[..., 2] - a[..., 1] > 4 * h) & (a[..., 0] > 4 * h)
    settled = settled.repeat_interleave(4, 1).reshape(M, K)
    assert float(settled.double().mean()) > 0.5
    steps = torch.eye(K, dtype=torch.float64, device=DEV) * h
    for m in range(M):
        up, down = ao.sparsify(x[m] + steps), ao.sparsify(x[m] - steps)
        num = ((up - down) @ G[m].double()) / (2 * h)
        off = (num - dX[m]).abs()[settled[m]]
        # the difference's own error: h^2 curvature and 64-bit cancellation, both below 1e-8
        assert bool((off <= tol[m][settled[m]] + 1e-8).all())


def test_a_block_that_is_not_finite_marks_its_row():
    X = normal(1, 4, 256)
    X[1, 70] = float("inf")
    q, e, _ = checkpoint(X, lynx.LYNX_CKPT8_INT8)
    dX = lynx.lynx_sparsify_backward(normal(2, 4, 256), q, e)
    assert not bool(dX[1].isfinite().any()) and bool(dX[[0, 2, 3]].isfinite().all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_what_the_selection_drops_is_not_read(fmt):
    """G may hold anything where the selection drops the value, and a kept zero
    (a row of zeros keeps its first two places) has sign 0."""
    M, K = 5, 320
    X = heavy(3, M, K)
    X[2] = 0
    q, e, x = checkpoint(X, fmt)
    G = normal(4, M, K)
    want = lynx.lynx_sparsify_backward(G, q, e)
    kept = ao.keep(x) > 0
    for bad in (float("inf"), float("-inf"), float("nan"), torch.finfo(torch.bfloat16).min):
        assert torch.equal(lynx.lynx_sparsify_backward(torch.where(kept, G, bad), q, e), want)
    assert torch.equal(want[2], torch.where(kept[2], G[2], 0))


def test_graph_replay_and_streams():
    M, N, K, r = 300, 520, 640, 64
    q, e, x = checkpoint(heavy(1, M, K), lynx.LYNX_CKPT8_E4M3)
    dY, A, B, G = normal(2, M, N), normal(3, r, K), normal(4, N, r), normal(5, M, K)

    def step(stream=None):
        dA, dB, dT = lynx.lynx_lora_backward(dY, q, e, A, B, stream=stream)
        return dA, dB, dT, lynx.lynx_sparsify_backward(G, q, e, dT, A, stream=stream)

    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [step(s) for _ in range(10) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1 = step()
    with torch.cuda.graph(g2):
        o2 = step()
    dY.copy_(normal(20, M, N))
    g1.replay()
    g2.replay()
    torch.cuda.synchronize()
    want = step()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, o1, o2))


@pytest.mark.parametrize("fmt", FORMATS)
def test_training_step_then_serving(fmt):
    """The operators as they are used together: forward through the sparse
    layer, X kept in 8 bits, the backward pass, an adapter step, the frozen
    weight to 4 bits, and one token through it with the new adapter."""
    M, N, K, r = 260, 576, 640, 64  # N % 64 == 0: the sum of the transposed products
    X, W, bias = heavy(1, M, K), normal(2, N, K, std=0.04), normal(3, N, std=0.02)
    A, B = normal(4, r, K, std=0.05), normal(5, N, r, std=0.05)
    Wt = W.t().contiguous()
    Y = lynx.lynx_linear(X, W, bias, A, B)
    q, e, x = checkpoint(X, fmt)
    dY = (Y.float() * 1e-2).bfloat16()
    dA, dB, dT = lynx.lynx_lora_backward(dY, q, e, A, B)
    G = lynx.lynx_linear_dense(dY, Wt)
    dX = lynx.lynx_sparsify_backward(G, q, e, dT, A)
    ref = ao.lora_backward(dY, x, A, B)
    for name, got in (("dA", dA), ("dB", dB), ("dT", dT)):
        within(got, *ref[name], name)
    within(dX, *ao.sparsify_backward(G, x, dT, A))
    # G itself: one rounding of a sum of N products
    g, gabs = dY.double() @ W.double(), dY.double().abs() @ W.double().abs()
    within(G, g, ao.BF * g.abs() + (N + 16) * ao.F32 * gabs + ao.TINY)
    # the dense path's gradient of X is the layer itself with the transposed operands
    dXd = lynx.lynx_linear_dense(dY, Wt, None, B.t().contiguous(), A.t().contiguous())
    d = g + dT.double() @ A.double()
    dabs = gabs + ref["dT"][0].abs() @ A.double().abs()
    within(dXd, d, ao.BF * d.abs() + (N + r + 16) * ao.F32 * dabs
           + 2.1 * ref["dT"][1] @ A.double().abs() + ao.TINY)
    A2 = (A.float() - 0.1 * dA.float()).bfloat16()
    B2 = (B.float() - 0.1 * dB.float()).bfloat16()
    Wq, sc, ze = lynx.lynx_w4_quantize(W, 128, True)
    token = X[:1].contiguous()
    y = lynx.lynx_linear_w4(token, Wq, sc, ze, bias, A2, B2, act=lynx.LYNX_ACT_GELU_TANH)
    v = ao.w4_values(*ao.w4_quantize(W, 128, True))
    within(y, *ao.linear_w4(token, v, bias, A2, B2, True))


def test_bindings_refuse():
    M, N, K, r = 8, 64, 128, 16
    q, e, _ = checkpoint(normal(1, M, K), lynx.LYNX_CKPT8_INT8)
    dY, A, B, G = normal(2, M, N), normal(3, r, K), normal(4, N, r), normal(5, M, K)
    with pytest.raises(ValueError):
        lynx.lynx_lora_backward(dY[:4], q, e, A, B)
    with pytest.raises(ValueError):
        lynx.lynx_lora_backward(dY.t().contiguous().t(), q, e, A, B)
    with pytest.raises(lynx.LynxError):
        lynx.lynx_lora_backward(dY, q, e, normal(3, 24, K), normal(4, N, 24))
    with pytest.raises(ValueError):
        lynx.lynx_lora_backward(dY, q, e, A, B[:8])
    with pytest.raises(lynx.LynxError):
        lynx.lynx_lora_backward(dY, q, e, A, B, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        lynx.lynx_sparsify_backward(G, q, e, A=A)
    with pytest.raises(TypeError):
        lynx.lynx_sparsify_backward(G.float(), q, e)
    with pytest.raises(ValueError):
        lynx.lynx_sparsify_backward(G, q, e[:4])


@pytest.mark.parametrize("op", ["lora", "sparsify"])
def test_waits_that_run_out_are_reported(op):
    """With the loads switched off the kernels' bounded waits run out, the call's
    stream says so, and the next call is right."""
    M, N, K, r = 200, 264, 320, 32
    q, e, x = checkpoint(heavy(1, M, K), lynx.LYNX_CKPT8_INT8)
    dY, A, B, G, dT = normal(2, M, N), normal(3, r, K), normal(4, N, r), normal(5, M, K), normal(6, M, r)

    def call():
        if op == "lora":
            return lynx.lynx_lora_backward(dY, q, e, A, B)[2]
        return lynx.lynx_sparsify_backward(G, q, e, dT, A)

    lynx.lynx_check_error()
    lynx.lynx_debug_set_stall(True)
    try:
        call()
    finally:
        lynx.lynx_debug_set_stall(False)
    st, code = lynx.lynx_check_error()
    assert st == lynx.LYNX_ERR_DEVICE_TIMEOUT and code != 0
    got = call()
    st, _ = lynx.lynx_check_error()
    assert st == lynx.LYNX_OK
    within(got, *(ao.lora_backward(dY, x, A, B)["dT"] if op == "lora" else ao.sparsify_backward(G, x, dT, A)))
