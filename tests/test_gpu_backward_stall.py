"""The selection gradient's give-up path: with the loads switched off every wait of
every block runs out, and the call ends, says so, and leaves nothing behind that the
next calls on the stream could meet."""
import pytest
import torch

from activation_sparse_gemm_lynx_b200 import lynx

import adapter_oracle as ao
from test_gpu_w4 import normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,r", [(1, 64, 16), (300, 1088, 0), (300, 1088, 64), (2049, 2048, 256)])
def test_a_stalled_call_ends_and_the_next_are_right(M, K, r):
    torch.cuda.set_device(0)
    q, e = lynx.lynx_ckpt8_store(normal(1, M, K))
    G = normal(2, M, K)
    dT, A = (normal(3, M, r), normal(4, r, K, std=0.2)) if r else (None, None)
    want = lynx.lynx_sparsify_backward(G, q, e, dT, A)
    x = ao.ckpt8_values(q.double(), e.long(), True)
    ref, tol = ao.sparsify_backward(G, x, dT, A)
    assert bool(((want.double() - ref).abs() <= tol).all())
    assert lynx.lynx_check_error()[0] == lynx.LYNX_OK
    lynx.lynx_debug_set_stall(True)
    try:
        lynx.lynx_sparsify_backward(G, q, e, dT, A)
    finally:
        lynx.lynx_debug_set_stall(False)
    after = [lynx.lynx_sparsify_backward(G, q, e, dT, A) for _ in range(3)]
    st, code = lynx.lynx_check_error()
    assert st == lynx.LYNX_ERR_DEVICE_TIMEOUT and code != 0
    assert all(torch.equal(t, want) for t in after)
    assert lynx.lynx_check_error()[0] == lynx.LYNX_OK
