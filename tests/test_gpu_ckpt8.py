"""The 8-bit checkpoint against its definition in 64 bits: equal, bit for bit."""
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
    torch.cuda.synchronize()


def check(X, fmt):
    M, K = X.shape
    int8 = fmt == lynx.LYNX_CKPT8_INT8
    raws = [guarded((M, K), torch.int8 if int8 else torch.float8_e4m3fn), guarded((M, K // 32), torch.uint8),
            guarded((M, K), torch.bfloat16)]
    (_, q), (_, e), (_, back) = raws
    lynx.lynx_ckpt8_store(X, fmt, q=q, e=e)
    lynx.lynx_ckpt8_restore(q, e, X=back)
    wq, we = ao.ckpt8_store(X, int8)
    assert torch.equal(e.long(), we)
    assert torch.equal(q.float().double(), wq)
    want = ao.ckpt8_values(wq, we, int8)
    assert torch.equal(back.double().nan_to_num(nan=12345.0), want.nan_to_num(nan=12345.0))
    assert all(intact(r, t) for r, t in raws)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K", [(1, 64), (2, 128), (3, 576), (300, 192), (257, 1088), (1, 12288), (1031, 4160)])
def test_store_and_restore(M, K, fmt):
    X = normal(M + K, M, K)
    large = normal(7, M, K).float() < -1.4  # a heavy tail
    check(torch.where(large, X, X * 0.05), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_bf16_value(fmt):
    """All 65536 bit patterns, each as its block's largest and beside others."""
    bits = torch.arange(65536, device=DEV, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    alone = torch.zeros(65536, 64, dtype=torch.bfloat16, device=DEV)
    alone[:, 13] = bits
    alone[:, 40] = bits.abs()
    check(alone, fmt)
    check(bits.view(256, 256).contiguous(), fmt)   # sorted: like magnitudes together
    g = torch.Generator(device=DEV).manual_seed(3)
    finite = bits[torch.isfinite(bits)]
    pick = torch.randint(0, finite.numel(), (512, 256), generator=g, device=DEV)
    check(finite[pick], fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_blocks_that_are_not_finite(fmt):
    X = normal(1, 4, 128)
    X[0, 3], X[1, 40], X[2, 127] = float("inf"), float("nan"), float("-inf")
    check(X, fmt)
    q, e = lynx.lynx_ckpt8_store(X, fmt)
    back = lynx.lynx_ckpt8_restore(q, e)
    assert e.eq(255).sum() == 3 and back.isnan().sum() == 96 and bool(back[3].isfinite().all())


def test_capture_and_other_stream():
    X = normal(5, 300, 576)
    want = lynx.lynx_ckpt8_restore(*lynx.lynx_ckpt8_store(X))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q, e = lynx.lynx_ckpt8_store(X, stream=s)
    back = lynx.lynx_ckpt8_restore(q, e, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(back, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        back = lynx.lynx_ckpt8_restore(*lynx.lynx_ckpt8_store(X))
    X.copy_(normal(6, 300, 576))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(back, lynx.lynx_ckpt8_restore(*lynx.lynx_ckpt8_store(X)))


def test_bindings_refuse():
    X = normal(1, 4, 128)
    q, e = lynx.lynx_ckpt8_store(X)
    with pytest.raises(lynx.LynxError):
        lynx.lynx_ckpt8_store(X, 5)
    with pytest.raises(lynx.LynxError):
        lynx.lynx_ckpt8_store(normal(1, 4, 96))
    with pytest.raises(TypeError):
        lynx.lynx_ckpt8_restore(q.view(torch.uint8), e)
    with pytest.raises(ValueError):
        lynx.lynx_ckpt8_restore(q, e[:, :2])
    with pytest.raises(ValueError):
        lynx.lynx_ckpt8_restore(q.t(), e)
