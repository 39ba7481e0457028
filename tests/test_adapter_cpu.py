"""Host-side checks of the 4-bit weight, checkpoint and backward entry points:
sizes, refusals (nothing is launched, so fake addresses do), and the formulas of
the tests' own 64-bit oracle against differences."""
import ctypes

import pytest
import torch

from activation_sparse_gemm_lynx_b200 import build as lynx_build
from activation_sparse_gemm_lynx_b200 import lynx

import adapter_oracle as ao

P = 0x10000000  # never dereferenced
BIG = 1 << 34


def vp(x):
    return ctypes.c_void_p(x)


@pytest.fixture(scope="module")
def lib():
    lynx_build.build()
    return lynx.library()


def call(lib, name, order, kw):
    return getattr(lib, name)(*[vp(kw[k]) if k in PTRS else kw[k] for k in order])


PTRS = {"W", "Wq", "scales", "zeros", "X", "bias", "A", "B", "Y", "ws", "q", "e", "dY", "dA", "dB", "dT", "G", "dX",
        "stream"}

ENTRY = {
    "lynx_w4_quantize": (["W", "N", "K", "group", "Wq", "scales", "zeros", "stream"],
                         dict(W=P, N=64, K=256, group=64, Wq=P, scales=P, zeros=None, stream=None)),
    "lynx_w4_dequantize": (["Wq", "scales", "zeros", "N", "K", "group", "W", "stream"],
                           dict(W=P, N=64, K=256, group=64, Wq=P, scales=P, zeros=P, stream=None)),
    "lynx_linear_w4": (["X", "Wq", "scales", "zeros", "bias", "A", "B", "M", "N", "K", "r", "group", "act", "Y", "ws",
                        "bytes", "stream"],
                       dict(X=P, Wq=P, scales=P, zeros=None, bias=None, A=P, B=P, M=4, N=64, K=256, r=16, group=64,
                            act=0, Y=P, ws=P, bytes=BIG, stream=None)),
    "lynx_ckpt8_store": (["X", "M", "K", "format", "q", "e", "stream"],
                         dict(X=P, M=4, K=256, format=0, q=P, e=P, stream=None)),
    "lynx_ckpt8_restore": (["q", "e", "M", "K", "format", "X", "stream"],
                           dict(X=P, M=4, K=256, format=1, q=P, e=P, stream=None)),
    "lynx_lora_backward": (["dY", "q", "e", "A", "B", "M", "N", "K", "r", "format", "dA", "dB", "dT", "ws", "bytes",
                            "stream"],
                           dict(dY=P, q=P, e=P, A=P, B=P, M=4, N=64, K=256, r=16, format=0, dA=P, dB=P, dT=None, ws=P,
                                bytes=BIG, stream=None)),
    "lynx_sparsify_backward": (["G", "q", "e", "dT", "A", "M", "K", "r", "format", "dX", "ws", "bytes", "stream"],
                               dict(G=P, q=P, e=P, dT=None, A=None, M=4, K=256, r=0, format=0, dX=P, ws=P, bytes=BIG,
                                    stream=None)),
}

for _order, _kw in ENTRY.values():  # buffers of their own
    for _i, _k in enumerate(_order):
        if _k in PTRS and _kw[_k] is not None:
            _kw[_k] = P + (_i << 36)

INVALID, SHAPE, ALIGN, SMALL = (lynx.LYNX_ERR_INVALID_ARG, lynx.LYNX_ERR_UNSUPPORTED_SHAPE, lynx.LYNX_ERR_MISALIGNED,
                                lynx.LYNX_ERR_WORKSPACE_TOO_SMALL)

BAD = [
    ("lynx_w4_quantize", dict(W=None), INVALID), ("lynx_w4_quantize", dict(Wq=None), INVALID),
    ("lynx_w4_quantize", dict(scales=None), INVALID), ("lynx_w4_quantize", dict(group=16), SHAPE),
    ("lynx_w4_quantize", dict(group=0), SHAPE), ("lynx_w4_quantize", dict(K=192, group=128), SHAPE),
    ("lynx_w4_quantize", dict(N=12), SHAPE), ("lynx_w4_quantize", dict(N=0), SHAPE),
    ("lynx_w4_quantize", dict(K=96), SHAPE), ("lynx_w4_quantize", dict(K=0), SHAPE),
    ("lynx_w4_quantize", dict(zeros=P + 8), ALIGN), ("lynx_w4_quantize", dict(W=P + 2), ALIGN),
    ("lynx_w4_dequantize", dict(W=None), INVALID), ("lynx_w4_dequantize", dict(N=-8), SHAPE),
    ("lynx_w4_dequantize", dict(scales=P + 4), ALIGN), ("lynx_w4_dequantize", dict(group=256), SHAPE),
    ("lynx_linear_w4", dict(X=None), INVALID), ("lynx_linear_w4", dict(Y=None), INVALID),
    ("lynx_linear_w4", dict(Wq=None), INVALID), ("lynx_linear_w4", dict(scales=None), INVALID),
    ("lynx_linear_w4", dict(act=2), INVALID), ("lynx_linear_w4", dict(A=None), INVALID),
    ("lynx_linear_w4", dict(B=None), INVALID), ("lynx_linear_w4", dict(ws=None), INVALID),
    ("lynx_linear_w4", dict(M=0), SHAPE), ("lynx_linear_w4", dict(M=33), SHAPE),
    ("lynx_linear_w4", dict(N=60), SHAPE), ("lynx_linear_w4", dict(K=72), SHAPE),
    ("lynx_linear_w4", dict(group=96), SHAPE), ("lynx_linear_w4", dict(r=24), SHAPE),
    ("lynx_linear_w4", dict(r=0), SHAPE), ("lynx_linear_w4", dict(r=272), SHAPE),
    ("lynx_linear_w4", dict(A=None, B=None, r=17), SHAPE),
    ("lynx_linear_w4", dict(bytes=4 * 16 * 4 - 1), SMALL), ("lynx_linear_w4", dict(bias=P + 2), ALIGN),
    ("lynx_linear_w4", dict(ws=P + 8), ALIGN),
    ("lynx_ckpt8_store", dict(X=None), INVALID), ("lynx_ckpt8_store", dict(format=2), INVALID),
    ("lynx_ckpt8_store", dict(format=-1), INVALID), ("lynx_ckpt8_store", dict(M=0), SHAPE),
    ("lynx_ckpt8_store", dict(K=32), SHAPE), ("lynx_ckpt8_store", dict(e=P + 1), ALIGN),
    ("lynx_ckpt8_restore", dict(e=None), INVALID), ("lynx_ckpt8_restore", dict(K=100), SHAPE),
    ("lynx_ckpt8_restore", dict(X=P + 8), ALIGN),
    ("lynx_lora_backward", dict(dY=None), INVALID), ("lynx_lora_backward", dict(A=None), INVALID),
    ("lynx_lora_backward", dict(dB=None), INVALID), ("lynx_lora_backward", dict(ws=None), INVALID),
    ("lynx_lora_backward", dict(format=3), INVALID), ("lynx_lora_backward", dict(r=8), SHAPE),
    ("lynx_lora_backward", dict(N=4), SHAPE), ("lynx_lora_backward", dict(M=-1), SHAPE),
    ("lynx_lora_backward", dict(dT=P + 2), ALIGN), ("lynx_lora_backward", dict(bytes=0), SMALL),
    ("lynx_sparsify_backward", dict(G=None), INVALID), ("lynx_sparsify_backward", dict(dT=P), INVALID),
    ("lynx_sparsify_backward", dict(A=P, r=16), INVALID), ("lynx_sparsify_backward", dict(dT=P, A=P, r=0), SHAPE),
    ("lynx_sparsify_backward", dict(r=7), SHAPE), ("lynx_sparsify_backward", dict(K=65), SHAPE),
    ("lynx_sparsify_backward", dict(M=0), SHAPE), ("lynx_sparsify_backward", dict(dX=P + 2), ALIGN),
    ("lynx_sparsify_backward", dict(dX=None), INVALID), ("lynx_sparsify_backward", dict(format=2), INVALID),
    ("lynx_sparsify_backward", dict(ws=None), INVALID), ("lynx_sparsify_backward", dict(bytes=0), SMALL),
]


@pytest.mark.parametrize("name,change,want", BAD)
def test_refusals(lib, name, change, want):
    order, kw = ENTRY[name]
    assert call(lib, name, order, {**kw, **change}) == want


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses: only where no kernel can start")
@pytest.mark.parametrize("name", sorted(ENTRY))
def test_good_arguments_pass_the_checks(lib, name):
    order, kw = ENTRY[name]
    assert call(lib, name, order, kw) == lynx.LYNX_ERR_CUDA  # no device here


def test_sizes(lib):
    assert lynx.lynx_w4_bytes(64, 256) == 64 * 128
    assert lynx.lynx_linear_w4_max_rows() == 32
    assert lynx.lynx_linear_w4_workspace_bytes(4, 64, 256, 0) == 0
    assert lynx.lynx_linear_w4_workspace_bytes(4, 64, 256, 16) >= 4 * 16 * 4
    assert lynx.lynx_ckpt8_exponent_bytes(7, 320) == 70
    assert lynx.lynx_lora_backward_workspace_bytes(0, 64, 256, 16) == 0
    assert lynx.lynx_lora_backward_workspace_bytes(300, 1000, 576, 16) > 0
    assert lynx.lynx_sparsify_backward_workspace_bytes(5, 60) == 0
    assert lynx.lynx_sparsify_backward_workspace_bytes(5, 64) >= 5 * 8


def test_bindings_refuse_cpu_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, e = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError):
        lynx.lynx_w4_quantize(x, 64)
    with pytest.raises(ValueError):
        lynx.lynx_ckpt8_store(x)
    with pytest.raises(ValueError):
        lynx.lynx_ckpt8_restore(q, e)
    with pytest.raises(ValueError):
        lynx.lynx_sparsify_backward(x, q, e)
    with pytest.raises(ValueError):
        lynx.lynx_lora_backward(x, q, e, x, x)
    with pytest.raises(ValueError):
        lynx.lynx_linear_w4(x, torch.zeros(8, 32, dtype=torch.uint8), x[:1, :8])


OUTPUTS = {
    "lynx_w4_quantize": ["Wq", "scales", "zeros"], "lynx_w4_dequantize": ["W"], "lynx_linear_w4": ["Y", "ws"],
    "lynx_ckpt8_store": ["q", "e"], "lynx_ckpt8_restore": ["X"],
    "lynx_lora_backward": ["dA", "dB", "dT", "ws"], "lynx_sparsify_backward": ["dX", "ws"],
}


@pytest.mark.parametrize("name", sorted(ENTRY))
def test_an_output_overlaps_no_other_buffer(lib, name):
    order, kw = ENTRY[name]
    kw = {**kw, **({"dT": P + (20 << 36), "A": P + (21 << 36), "r": 16} if name == "lynx_sparsify_backward" else {}),
          **{k: P + (22 + i << 36) for i, k in enumerate(["zeros", "bias", "dT"]) if k in kw and kw[k] is None}}
    buffers = [k for k in order if k in PTRS and k != "stream"]
    for out in OUTPUTS[name]:
        for other in buffers:
            if other != out:
                # from its start, and from its second 16 bytes on
                assert call(lib, name, order, {**kw, out: kw[other]}) == INVALID, (out, other)
                assert call(lib, name, order, {**kw, out: kw[other] + 16}) == INVALID, (out, other)
    # inputs may be the same buffer
    if name == "lynx_lora_backward" and not torch.cuda.is_available():
        assert call(lib, name, order, {**kw, "N": 256, "M": 4, "A": kw["B"]}) == lynx.LYNX_ERR_CUDA


# ---- the oracle's formulas --------------------------------------------------


def test_sparsify_gradient_against_differences():
    g = torch.Generator().manual_seed(5)
    x = torch.randn(3, 64, generator=g, dtype=torch.float64)
    G = torch.randn(3, 64, generator=g, dtype=torch.float64)
    dX, _ = ao.sparsify_backward(G, x)
    h = 1e-6  # far below the gaps between magnitudes, so the selection stays
    a = x.abs().reshape(3, -1, 4).sort(dim=2).values
    assert float((a[..., 1:] - a[..., :-1]).min()) > 10 * h and float(a.min()) > 10 * h
    num = torch.empty_like(x)
    for m in range(3):
        for k in range(64):
            d = torch.zeros_like(x)
            d[m, k] = h
            num[m, k] = ((G * ao.sparsify(x + d)).sum() - (G * ao.sparsify(x - d)).sum()) / (2 * h)
    assert float((num - dX).abs().max()) < 1e-7


def test_sparsify_gradient_keeps_a_zero_row_finite():
    x = torch.zeros(2, 64, dtype=torch.float64)
    G = torch.ones(2, 64, dtype=torch.float64)
    dX, _ = ao.sparsify_backward(G, x)
    assert torch.equal(dX, ao.keep(x)) and float(dX.sum()) == 64


def test_lora_gradients_against_differences():
    g = torch.Generator().manual_seed(6)
    f = dict(generator=g, dtype=torch.float64)
    x, A, B, dY = torch.randn(5, 64, **f), torch.randn(16, 64, **f), torch.randn(8, 16, **f), torch.randn(5, 8, **f)
    got = ao.lora_backward(dY, x, A, B)

    def loss(a, b):
        return float((dY * ((x @ a.t()) @ b.t())).sum())

    for which, p in (("dA", A), ("dB", B)):
        for i, j in ((0, 0), (3, 5), (7, 15)):
            d = torch.zeros_like(p)
            d[i, j] = 0.5  # linear in each adapter matrix: any step will do
            up = loss(A + d, B) - loss(A - d, B) if which == "dA" else loss(A, B + d) - loss(A, B - d)
            assert abs(up - float(got[which][0][i, j])) < 1e-9


@pytest.mark.parametrize("int8", [True, False])
def test_checkpoint_error_bounds(int8):
    """The bounds include/lynx.h states, and exactness of the values in bf16."""
    g = torch.Generator().manual_seed(7)
    x = torch.randn(64, 256, generator=g) * torch.exp2(torch.randint(-30, 30, (64, 1), generator=g).float())
    x[0] = torch.randn(256, generator=g) * 2.0 ** -130
    x[1, ::7] = 3.3e38
    x = x.bfloat16()
    q, e = ao.ckpt8_store(x, int8)
    v = ao.ckpt8_values(q, e, int8)
    assert torch.equal(v, v.bfloat16().double())
    top = x.double().abs().reshape(64, -1, 32).amax(2).repeat_interleave(32, 1)
    off = (v - x.double()).abs()
    if int8:
        assert bool((off <= 2.0 ** -7 * top).all())
    else:
        fine = (x.double().abs() >= 2.0 ** -13 * top) & (top < 2.0 ** 127) & (top > 2.0 ** -119)
        assert bool((off <= 2.0 ** -4 * x.double().abs())[fine].all())
