"""Host-side checks of the layer norm, residual and activation-gradient entry points: what
is refused is refused before the device is touched."""
import ctypes

import pytest
import torch

from activation_sparse_gemm_lynx_b200 import build as lynx_build
from activation_sparse_gemm_lynx_b200 import lynx

P = 0x100000000  # fake, never dereferenced
GAP = 1 << 34
OK = (lynx.LYNX_OK, lynx.LYNX_ERR_CUDA)  # the checks passed; without a device the launch fails


@pytest.fixture(scope="module")
def lib():
    lynx_build.build()
    return lynx.library()


def at(i, off=0):
    """The i-th of fake buffers that lie far apart"""
    return ctypes.c_void_p(P + i * GAP + off)


NO_DEVICE = not torch.cuda.is_available()
needs_no_device = pytest.mark.skipif(not NO_DEVICE, reason="accepted calls would run on fake addresses")


def norm(lib, X=at(1), w=at(2), b=at(3), M=300, K=576, eps=1e-6, Y=at(4), mean=at(5), rstd=at(6)):
    return lib.lynx_layer_norm(X, w, b, M, K, eps, Y, mean, rstd, None)


def test_layer_norm_refusals(lib):
    assert lynx.lynx_layer_norm_max_cols() == 32768
    assert norm(lib, X=None) == lynx.LYNX_ERR_INVALID_ARG
    assert norm(lib, Y=None) == lynx.LYNX_ERR_INVALID_ARG
    assert norm(lib, mean=None) == lynx.LYNX_ERR_INVALID_ARG
    assert norm(lib, rstd=None) == lynx.LYNX_ERR_INVALID_ARG
    for eps in (-1e-6, float("nan"), float("inf")):
        assert norm(lib, eps=eps) == lynx.LYNX_ERR_INVALID_ARG
    for M, K in ((0, 576), (-1, 576), (300, 0), (300, 4), (300, 100), (300, 32776), (1 << 31, 576)):
        assert norm(lib, M=M, K=K) == lynx.LYNX_ERR_UNSUPPORTED_SHAPE
    for kw in (dict(X=at(1, 8)), dict(w=at(2, 2)), dict(b=at(3, 4)), dict(Y=at(4, 8)), dict(mean=at(5, 4))):
        assert norm(lib, **kw) == lynx.LYNX_ERR_MISALIGNED
    for kw in (dict(Y=at(1)), dict(Y=at(1, 16)), dict(Y=at(2)), dict(mean=at(1)), dict(rstd=at(5)), dict(mean=at(4))):
        assert norm(lib, **kw) == lynx.LYNX_ERR_INVALID_ARG


@needs_no_device
def test_layer_norm_accepts(lib):
    for kw in ({}, dict(w=None), dict(b=None), dict(mean=None, rstd=None), dict(eps=0.0), dict(M=1, K=8), dict(K=32768)):
        assert norm(lib, **kw) in OK


def norm_backward(lib, dY=at(1), X=at(2), mean=at(3), rstd=at(4), w=at(5), dR=at(6), M=3000, K=576, dX=at(7), dw=at(8), db=at(9),
                  ws=at(10), ws_bytes=1 << 30):
    return lib.lynx_layer_norm_backward(dY, X, mean, rstd, w, dR, M, K, dX, dw, db, ws, ws_bytes, None)


def test_layer_norm_backward_refusals(lib):
    for name in ("dY", "X", "mean", "rstd", "dX", "ws"):
        assert norm_backward(lib, **{name: None}) == lynx.LYNX_ERR_INVALID_ARG, name
    for M, K in ((0, 576), (300, 4), (300, 100), (300, 32776)):
        assert norm_backward(lib, M=M, K=K) == lynx.LYNX_ERR_UNSUPPORTED_SHAPE
        assert lynx.lynx_layer_norm_backward_workspace_bytes(M, K) == 0
    for i, name in enumerate(("dY", "X", "mean", "rstd", "w", "dR", "dX", "dw", "db", "ws")):
        assert norm_backward(lib, **{name: at(i + 1, 8)}) == lynx.LYNX_ERR_MISALIGNED, name
    for K in (8, 576, 4096, 8192, 8200, 32768):
        need = lynx.lynx_layer_norm_backward_workspace_bytes(3000, K)
        assert need >= 2 * K * 4
        assert norm_backward(lib, M=3000, K=K, ws_bytes=need - 1) == lynx.LYNX_ERR_WORKSPACE_TOO_SMALL
        assert lynx.lynx_layer_norm_backward_workspace_bytes(1, K) == 0
    for kw in (dict(dX=at(1)), dict(dX=at(2)), dict(dX=at(5)), dict(dX=at(6, 16)), dict(dw=at(9)), dict(dw=at(6)), dict(db=at(6)),
               dict(ws=at(6)), dict(ws=at(7)), dict(db=at(5)), dict(dw=at(3)), dict(dY=at(6), dX=at(6)), dict(X=at(6), dX=at(6))):
        assert norm_backward(lib, **kw) == lynx.LYNX_ERR_INVALID_ARG


@needs_no_device
def test_layer_norm_backward_accepts(lib):
    for kw in ({}, dict(w=None), dict(dR=None), dict(dX=at(6)), dict(dw=None), dict(db=None), dict(K=32768),
               dict(dw=None, db=None, ws=None, ws_bytes=0), dict(M=1, ws=None, ws_bytes=0)):
        assert norm_backward(lib, **kw) in OK


def residual(lib, X=at(1), W=at(2), bias=at(3), A=at(4), B=at(5), R=at(6), M=300, N=1000, K=576, r=16, skip=0, act=1, Y=at(7),
             Z=at(8), ws=at(9), ws_bytes=1 << 30):
    return lib.lynx_linear_residual(X, W, bias, A, B, R, M, N, K, r, skip, act, Y, Z, ws, ws_bytes, None)


def test_linear_residual_refusals(lib):
    for name in ("X", "W", "A", "B", "Y", "ws"):
        assert residual(lib, **{name: None}) == lynx.LYNX_ERR_INVALID_ARG, name
    for act in (-1, 2):
        assert residual(lib, act=act) == lynx.LYNX_ERR_INVALID_ARG
    for kw in (dict(M=0), dict(N=12), dict(K=100), dict(r=24), dict(M=(1 << 30) + 1)):
        assert residual(lib, **kw) == lynx.LYNX_ERR_UNSUPPORTED_SHAPE
    for i, name in enumerate(("X", "W", "bias", "A", "B", "R", "Y", "Z", "ws")):
        assert residual(lib, **{name: at(i + 1, 8)}) == lynx.LYNX_ERR_MISALIGNED, name
    need = lynx.lynx_workspace_bytes(300, 1000, 576, 16)
    assert residual(lib, ws_bytes=need - 1) == lynx.LYNX_ERR_WORKSPACE_TOO_SMALL
    for kw in (dict(Y=at(1)), dict(Y=at(2)), dict(Y=at(6, 16)), dict(Z=at(6)), dict(Z=at(7)), dict(Y=at(8)), dict(ws=at(6)),
               dict(ws=at(7)), dict(Z=at(5)), dict(Y=at(6), Z=at(6)), dict(ws=at(8, 256)),
               dict(X=at(6), Y=at(6)), dict(W=at(6), Y=at(6)), dict(bias=at(6), Y=at(6))):
        assert residual(lib, **kw) == lynx.LYNX_ERR_INVALID_ARG, kw


@needs_no_device
def test_linear_residual_accepts(lib):
    for kw in ({}, dict(R=None), dict(Z=None), dict(R=None, Z=None), dict(Y=at(6)), dict(bias=None),
               dict(A=None, B=None, r=0, skip=1, ws=None, ws_bytes=0)):
        assert residual(lib, **kw) in OK, kw


def few(lib, X=at(1), Wq=at(2), scales=at(3), zeros=at(4), bias=at(5), A=at(6), B=at(7), R=at(8), M=3, N=1000, K=576, r=16,
        group=64, act=0, Y=at(9), ws=at(10), ws_bytes=1 << 20):
    return lib.lynx_linear_w4_residual(X, Wq, scales, zeros, bias, A, B, R, M, N, K, r, group, act, Y, ws, ws_bytes, None)


def test_linear_w4_residual_refusals(lib):
    assert few(lib, M=33) == lynx.LYNX_ERR_UNSUPPORTED_SHAPE
    assert few(lib, R=at(8, 8)) == lynx.LYNX_ERR_MISALIGNED
    for kw in (dict(Y=at(8, 16)), dict(ws=at(8)), dict(ws=at(8), Y=at(8)), dict(Y=at(1)), dict(act=2), dict(X=at(8), Y=at(8))):
        assert few(lib, **kw) == lynx.LYNX_ERR_INVALID_ARG, kw


def act_backward(lib, dY=at(1), Z=at(2), M=3000, N=1000, act=1, dZ=at(3), db=at(4), ws=at(5), ws_bytes=1 << 30):
    return lib.lynx_act_backward(dY, Z, M, N, act, dZ, db, ws, ws_bytes, None)


def test_act_backward_refusals(lib):
    for kw in (dict(dY=None), dict(Z=None), dict(dZ=None), dict(ws=None), dict(act=2), dict(act=-1),
               dict(act=0), dict(act=0, Z=None), dict(act=0, dZ=None), dict(act=0, Z=None, dZ=None, db=None)):
        assert act_backward(lib, **kw) == lynx.LYNX_ERR_INVALID_ARG, kw
    for M, N in ((0, 1000), (300, 0), (300, 12), (300, 1001)):
        assert act_backward(lib, M=M, N=N) == lynx.LYNX_ERR_UNSUPPORTED_SHAPE
        assert lynx.lynx_act_backward_workspace_bytes(M, N) == 0
    for i, name in enumerate(("dY", "Z", "dZ", "db", "ws")):
        assert act_backward(lib, **{name: at(i + 1, 4)}) == lynx.LYNX_ERR_MISALIGNED, name
    need = lynx.lynx_act_backward_workspace_bytes(3000, 1000)
    assert need >= 4000
    assert lynx.lynx_act_backward_workspace_bytes(300, 1000) == 0
    assert act_backward(lib, ws_bytes=need - 1) == lynx.LYNX_ERR_WORKSPACE_TOO_SMALL
    for kw in (dict(dZ=at(2)), dict(dZ=at(1, 16)), dict(db=at(1)), dict(ws=at(1)), dict(ws=at(3)), dict(db=at(3)), dict(db=at(5)),
               dict(Z=at(1), dZ=at(1))):
        assert act_backward(lib, **kw) == lynx.LYNX_ERR_INVALID_ARG, kw


@needs_no_device
def test_act_backward_accepts(lib):
    for kw in ({}, dict(dZ=at(1)), dict(db=None, ws=None, ws_bytes=0), dict(act=0, Z=None, dZ=None),
               dict(M=300, ws=None, ws_bytes=0)):
        assert act_backward(lib, **kw) in OK, kw


def test_bindings_refuse_before_the_device():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    for call in (lambda: lynx.lynx_layer_norm(x), lambda: lynx.lynx_layer_norm_backward(x, x, x, x),
                 lambda: lynx.lynx_act_backward(x, x), lambda: lynx.lynx_linear_residual(x, x),
                 lambda: lynx.lynx_linear_w4_residual(x, x, x)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()
    for call in (lambda: lynx.lynx_layer_norm(None), lambda: lynx.lynx_act_backward(None, x)):
        with pytest.raises(ValueError, match="is required"):
            call()
