"""Host-side checks of the selection gradient with the forward pass's metadata."""
import pytest
import torch

from activation_sparse_gemm_lynx_b200 import build as lynx_build
from activation_sparse_gemm_lynx_b200 import lynx

import selection_oracle as so
from test_adapter_cpu import ALIGN, ENTRY, INVALID, P, PTRS, SHAPE, SMALL, vp

_order, _kw = ENTRY["lynx_sparsify_backward"]
ORDER = _order[:3] + ["meta"] + _order[3:]
KW = {**_kw, "meta": P + (30 << 36)}


@pytest.fixture(scope="module")
def lib():
    lynx_build.build()
    return lynx.library()


def call(lib, **change):
    kw = {**KW, **change}
    return lib.lynx_sparsify_backward_meta(*[vp(kw[k]) if k in PTRS or k == "meta" else kw[k] for k in ORDER])


@pytest.mark.parametrize("change,want", [
    (dict(meta=None), INVALID), (dict(G=None), INVALID), (dict(dX=None), INVALID), (dict(format=2), INVALID),
    (dict(meta=P + (30 << 36) + 8), ALIGN), (dict(K=65), SHAPE), (dict(M=0), SHAPE), (dict(bytes=0), SMALL),
    (dict(dT=P + (31 << 36)), INVALID), (dict(dX=P + (30 << 36)), INVALID), (dict(ws=P + (30 << 36)), INVALID),
    # the metadata's last 16 bytes: 4 x 256 has 2 row blocks x 2 blocks of 2 KB
    (dict(dX=P + (30 << 36) + 4 * 2048 - 16), INVALID)])
def test_refusals(lib, change, want):
    assert call(lib, **change) == want


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses: only where no kernel can start")
def test_good_arguments_pass_the_checks(lib):
    assert call(lib) == lynx.LYNX_ERR_CUDA  # no device here
    assert call(lib, dX=P + (30 << 36) + 4 * 2048) == lynx.LYNX_ERR_CUDA


@pytest.mark.parametrize("M,K", [(1, 64), (300, 1088), (4608, 12288)])
def test_where_the_workspace_has_it(lib, M, K):
    at = lynx.lynx_workspace_meta_offset(M, K)
    assert at == -(-M * K // 256) * 256
    assert at + lynx.lynx_meta_bytes(M, K) <= lynx.lynx_workspace_bytes(M, 512, K, 16)
    assert lynx.lynx_workspace_meta_offset(0, K) == 0


def test_a_cpu_workspace_is_refused():
    with pytest.raises(ValueError):
        lynx.lynx_workspace_meta(torch.zeros(1 << 20, dtype=torch.uint8), 1, 64)


def test_the_formula_against_differences():
    """The 64-bit oracle with a selection that is not the values' own."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(3, 64, generator=g, dtype=torch.float64)
    G = torch.randn(3, 64, generator=g, dtype=torch.float64)
    m = torch.tensor([0.0, 1.0, 1.0, 0.0], dtype=torch.float64).repeat(3, 16)
    dX, _ = so.gradient(G, x, m)
    h = 1e-6
    num = torch.empty_like(x)
    for i in range(3):
        for k in range(64):
            d = torch.zeros_like(x)
            d[i, k] = h
            num[i, k] = ((G * so.layer(x + d, m)).sum() - (G * so.layer(x - d, m)).sum()) / (2 * h)
    assert float((num - dX).abs().max()) < 1e-7
