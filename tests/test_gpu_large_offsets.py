"""The 4-bit, checkpoint and backward calls where element offsets pass 32 bits
(rows at both ends hold values, the rest is zero), and as the first calls of a
process inside a stream capture."""
import subprocess
import sys
from pathlib import Path

import pytest
import torch

from activation_sparse_gemm_lynx_b200 import lynx

import adapter_oracle as ao
from test_gpu_w4 import DEV, normal

pytestmark = pytest.mark.gpu
M, K = 70016, 65600  # M * K = 4.59e9 elements
ENDS = [slice(0, 104), slice(M - 200, M)]


def ends(seed, cols, std=1.0):
    t = torch.zeros(M, cols, dtype=torch.bfloat16, device=DEV)
    for i, s in enumerate(ENDS):
        t[s] = normal(seed + i, s.stop - s.start, cols, std=std)
    return t


def rows(t):
    return torch.cat([t[s] for s in ENDS])


def within(got, ref, tol):
    assert float(((got.double() - ref).abs() / tol).max()) <= 1


@pytest.fixture(autouse=True)
def _room():
    torch.cuda.set_device(0)
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()
    st, code = lynx.lynx_check_error()
    assert st == lynx.LYNX_OK, (st, code)


def test_checkpoint_and_selection_gradient():
    X, G = ends(1, K), ends(3, K)
    q, e = lynx.lynx_ckpt8_store(X)
    few_q, few_e = lynx.lynx_ckpt8_store(rows(X))
    assert torch.equal(rows(q), few_q) and torch.equal(rows(e), few_e)
    assert not bool(q[ENDS[0].stop:ENDS[1].start].any())
    x = lynx.lynx_ckpt8_restore(q, e)
    assert torch.equal(rows(x), lynx.lynx_ckpt8_restore(few_q, few_e))
    values = rows(x).double()
    del X, x
    dT, A = ends(5, 16), normal(7, 16, K, std=0.2)
    dX = lynx.lynx_sparsify_backward(G, q, e, dT, A)
    within(rows(dX), *ao.sparsify_backward(rows(G), values, rows(dT), A))
    assert not bool(dX[ENDS[0].stop:ENDS[1].start].any())


@pytest.mark.parametrize("N,k", [(64, K), (K, 64)])
def test_adapter_gradients(N, k):
    r = 16
    q, e = lynx.lynx_ckpt8_store(ends(1, k))
    dY, A, B = ends(3, N), normal(5, r, k, std=k ** -0.5), normal(6, N, r, std=r ** -0.5)
    dA, dB, dT = lynx.lynx_lora_backward(dY, q, e, A, B)
    x = ao.ckpt8_values(rows(q).double(), rows(e).long(), True)
    want = ao.lora_backward(rows(dY), x, A, B)  # rows of zeros add nothing
    within(dA, *want["dA"])
    within(dB, *want["dB"])
    within(rows(dT), *want["dT"])


def test_weight_in_4_bits():
    N, group = M, 64
    W = ends(1, K, std=0.05)
    Wq, scales, zeros = lynx.lynx_w4_quantize(W, group, zero_points=True)
    few = lynx.lynx_w4_quantize(rows(W), group, zero_points=True)
    few_s, few_z = few[1], few[2]
    back = torch.cat([scales[:, s] for s in ENDS], 1), torch.cat([zeros[:, s] for s in ENDS], 1)
    assert torch.equal(rows(Wq), few[0]) and torch.equal(back[0], few_s) and torch.equal(back[1], few_z)
    del W
    w = lynx.lynx_w4_dequantize(Wq, scales, zeros)
    few_w = lynx.lynx_w4_dequantize(*few)
    assert torch.equal(rows(w), few_w) and not bool(w[ENDS[0].stop:ENDS[1].start].any())
    del w
    X = normal(9, 2, K)
    Y = lynx.lynx_linear_w4(X, Wq, scales, zeros)
    few_y = lynx.lynx_linear_w4(X, *few)
    got = torch.cat([Y[:, s] for s in ENDS], 1)
    # the same sums in another split
    size = X.double().abs() @ few_w.double().abs().t()
    within(got, few_y.double(), 2.0 ** -8 * few_y.double().abs() + 2 * 2.0 ** -24 * (K + 16) * size + 1e-30)
    assert not bool(Y[:, ENDS[0].stop:ENDS[1].start].any()) and N == Y.shape[1]


FIRST = """
import sys
import torch
from activation_sparse_gemm_lynx_b200 import lynx
torch.manual_seed(1)
X, dY = torch.randn(40, 256, device="cuda").bfloat16(), torch.randn(40, 136, device="cuda").bfloat16()
A, B = torch.randn(16, 256, device="cuda").bfloat16(), torch.randn(136, 16, device="cuda").bfloat16()
W = torch.randn(136, 256, device="cuda").bfloat16()
def step():
    q, e = lynx.lynx_ckpt8_store(X)
    x = lynx.lynx_ckpt8_restore(q, e)
    dA, dB, dT = lynx.lynx_lora_backward(dY, q, e, A, B)
    dX = lynx.lynx_sparsify_backward(x, q, e, dT, A)
    Wq, s, z = lynx.lynx_w4_quantize(W, 64, zero_points=True)
    return q, e, x, dA, dB, dT, dX, Wq, s, z, lynx.lynx_w4_dequantize(Wq, s, z), lynx.lynx_linear_w4(X[:3], Wq, s, z, None, A, B)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
for t in got:
    t.view(torch.uint8).fill_(0x5A)
graph.replay()
torch.cuda.synchronize()
want = step()
assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
assert lynx.lynx_check_error()[0] == lynx.LYNX_OK
print("equal")
"""


def test_first_calls_of_a_process_in_a_capture():
    run = subprocess.run([sys.executable, "-c", FIRST], cwd=Path(__file__).resolve().parent.parent, timeout=300,
                         capture_output=True, text=True)
    assert run.returncode == 0 and "equal" in run.stdout, run.stdout + run.stderr
