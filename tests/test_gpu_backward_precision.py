"""The adapter's gradients in the norm: they are off by the rounding of the results
alone, and what lies in the last, ragged block of a dimension counts."""
import pytest
import torch

from activation_sparse_gemm_lynx_b200 import lynx

import adapter_oracle as ao
from norms import rounded_once
from test_gpu_w4 import DEV, normal

pytestmark = pytest.mark.gpu
FORMATS = [lynx.LYNX_CKPT8_INT8, lynx.LYNX_CKPT8_E4M3]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    torch.cuda.set_device(0)
    lynx.library()
    yield
    st, code = lynx.lynx_check_error()
    assert st == lynx.LYNX_OK, (st, code)


def gradients(X, dY, A, B, fmt):
    q, e = lynx.lynx_ckpt8_store(X, fmt)
    x = ao.ckpt8_values(q.float().double(), e.long(), fmt == lynx.LYNX_CKPT8_INT8)
    dA, dB, dT = lynx.lynx_lora_backward(dY, q, e, A, B)
    return {"dT": dT, "dB": dB, "dA": dA}, ao.lora_backward(dY, x, A, B)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K,r", [(300, 1000, 576, 16), (2049, 72, 64, 80), (1025, 2056, 128, 192),
                                     (257, 136, 320, 208), (1000, 640, 256, 256), (300, 4104, 320, 256),
                                     (129, 520, 1088, 144), (4608, 1032, 512, 64), (70, 4096, 2048, 240),
                                     (1500, 2056, 4096, 112)])
def test_only_the_results_are_rounded(M, N, K, r, fmt):
    X = normal(M + K, M, K)
    X = torch.where(normal(M, M, K).float() < -1.4, X, X * 0.05)
    dY, A, B = normal(2, M, N, std=1e-3), normal(3, r, K, std=K ** -0.5), normal(4, N, r, std=N ** -0.5)
    got, ref = gradients(X, dY, A, B, fmt)
    for name in got:
        rounded_once(got[name], ref[name][0])


@pytest.mark.parametrize("M,N,K,r", [(2049, 72, 64, 80), (129, 1032, 4160, 64), (300, 264, 192, 256), (1, 8, 64, 16)])
@pytest.mark.parametrize("where", ["rows", "outputs", "columns", "rank"])
def test_the_last_block_counts(where, M, N, K, r):
    """All is zero but the last, ragged block of one dimension."""
    X, dY = normal(1, M, K), normal(2, M, N, std=1e-3)
    A, B = normal(3, r, K, std=K ** -0.5), normal(4, N, r, std=N ** -0.5)

    def last(t, dim, step):
        n = t.shape[dim]
        t.narrow(dim, 0, (n - 1) // step * step).zero_()

    if where == "rows":
        last(X, 0, 128)
    elif where == "outputs":
        last(dY, 1, 128)
    elif where == "columns":
        last(X, 1, 128)
    else:
        last(A, 0, 64)
        last(B, 1, 64)
    got, ref = gradients(X, dY, A, B, lynx.LYNX_CKPT8_INT8)
    for name in got:
        value, tol = ref[name]
        assert bool(value.any())
        assert bool(((got[name].double() - value).abs() <= tol).all())
        if value.count_nonzero() >= 500:
            rounded_once(got[name], value)


# Operands in 2 or 4 pieces and in single buffers, one or several inner blocks, with and
# without clusters and groups of them: the least work that the plan gives each form.
FORMS = [
    (129, 4104, 64, 96), (300, 12288, 64, 96), (129, 8, 64, 80), (1, 8, 64, 80), (1025, 12288, 64, 144),
    (129, 8, 64, 208), (1, 8, 64, 208), (129, 8, 64, 192), (1, 8, 64, 192), (129, 8, 64, 144), (1, 8, 64, 144),
    (1025, 9216, 64, 208), (4608, 2056, 64, 208), (2049, 4104, 64, 240), (4608, 4104, 64, 240),
    (513, 12288, 64, 256), (2049, 9216, 64, 144), (1025, 9216, 64, 192), (1025, 12288, 64, 192),
    (4608, 8, 2112, 208), (2049, 8, 12288, 208), (513, 8, 576, 208), (1, 8, 576, 208), (513, 8, 64, 144),
    (513, 8, 64, 192), (4608, 8, 4160, 80), (4608, 8, 12288, 80), (513, 8, 64, 80), (1025, 8, 64, 96),
    (2049, 8, 4160, 144), (2049, 8, 1088, 208), (300, 8, 64, 208)]


@pytest.mark.parametrize("i", range(len(FORMS)))
def test_every_form_of_the_passes(i):
    M, N, K, r = FORMS[i]
    X, dY = normal(1, M, K), normal(2, M, N, std=1e-3)
    A, B = normal(3, r, K, std=K ** -0.5), normal(4, N, r, std=N ** -0.5)
    got, ref = gradients(X, dY, A, B, FORMATS[i % 2])
    for name in got:
        value, tol = ref[name]
        assert bool(((got[name].double() - value).abs() <= tol).all())
        if value.numel() >= 500:
            rounded_once(got[name], value)
    again, _ = gradients(X, dY, A, B, FORMATS[i % 2])
    assert all(torch.equal(got[name], again[name]) for name in got)


@pytest.mark.parametrize("M,N,K,r", [(300, 1000, 576, 16), (129, 4104, 64, 96), (513, 12288, 64, 256),
                                     (2049, 8, 12288, 208), (1, 8, 576, 208)])
def test_dT_may_be_null_in_every_form(M, N, K, r):
    """The C call without dT: one pass over dY or two, with and without partial sums."""
    q, e = lynx.lynx_ckpt8_store(normal(1, M, K))
    dY, A, B = normal(2, M, N), normal(3, r, K), normal(4, N, r)
    want = lynx.lynx_lora_backward(dY, q, e, A, B)
    dA, dB = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = torch.empty(lynx.lynx_lora_backward_workspace_bytes(M, N, K, r), dtype=torch.uint8, device=DEV)
    p = lynx._ptr
    st = lynx.library().lynx_lora_backward(p(dY), p(q), p(e), p(A), p(B), M, N, K, r, lynx.LYNX_CKPT8_INT8, p(dA), p(dB),
                                           None, p(ws), ws.numel(), lynx._stream(None))
    assert st == lynx.LYNX_OK
    assert torch.equal(dA, want[0]) and torch.equal(dB, want[1])


def test_two_host_threads_on_their_own_streams():
    import threading

    M, N, K, r = 600, 1032, 1088, 144
    X, dY, G = normal(1, M, K), normal(2, M, N), normal(5, M, K)
    A, B = normal(3, r, K), normal(4, N, r)
    q, e = lynx.lynx_ckpt8_store(X)
    meta = lynx.lynx_sparsify(X)[1]

    def step(stream=None):
        dA, dB, dT = lynx.lynx_lora_backward(dY, q, e, A, B, stream=stream)
        return dA, dB, dT, lynx.lynx_sparsify_backward(G, q, e, dT, A, stream=stream, meta=meta)

    want = step()
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        torch.cuda.set_device(0)
        s = torch.cuda.Stream()
        for _ in range(20):
            got[i].append(step(s))
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(len(g) == 20 for g in got)
    assert all(torch.equal(a, b) for g in got for o in g for a, b in zip(o, want))


def test_an_infinite_gradient_stays_one():
    """Where a partial product overflows, the sum of its two halves is still infinite."""
    M, N, K, r = 2, 64, 64, 16
    X = torch.full((M, K), 1.0, dtype=torch.bfloat16, device=DEV)
    dY = torch.full((M, N), 3.0e38, dtype=torch.bfloat16, device=DEV)
    A, B = torch.ones(r, K, dtype=torch.bfloat16, device=DEV), torch.ones(N, r, dtype=torch.bfloat16, device=DEV)
    dA, dB, dT = lynx.lynx_lora_backward(dY, *lynx.lynx_ckpt8_store(X), A, B)
    for t in (dA, dB, dT):
        assert bool((t == float("inf")).all())
