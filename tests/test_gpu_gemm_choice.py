"""Which of the two GEMM kernels takes a layer, and that either gives the same bits.

Which one ran shows in the workspace: the CTA pairs join the pass's partials themselves and
keep a state word for every 32 rows there, at its end; the 1-CTA kernel leaves them alone.
"""
import pytest
import torch

import bench
from activation_sparse_gemm_lynx_b200 import lynx

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
POISON = 0x5A5A5A5A


def normal(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


def state_words(ws, M):
    words = ws.view(torch.int32)
    n = -(-M // 32)
    return words[words.numel() - -(-4 * n // 256) * 64:][:n]


def layer(M, N, K, r, seed=0):
    return (normal((M, K), seed + 1), normal((N, K), seed + 2, K ** -0.5), normal((N,), seed + 3),
            normal((r, K), seed + 4, 0.05) if r else None, normal((N, r), seed + 5, 0.05) if r else None)


# both sides of each border of the rule: rows, columns and K that the pairs take at all; more 128 x 128
# tiles than SMs; sparse, K past 2048, and past 1536 where tiles of 64 columns do not fit one round and
# at most 32 ranks are to be joined
SHAPES = [(128, 20000, 256), (129, 20000, 256), (20000, 248, 128), (20000, 256, 128), (1300, 2056, 192), (1300, 2056, 256),
          (512, 4736, 256), (512, 4744, 256), (300, 520, 2048), (300, 520, 2176), (1000, 2304, 1536), (1000, 2304, 1664),
          (1000, 2304, 2048), (1000, 1152, 2048), (1000, 1160, 2048)]


@pytest.mark.parametrize("r", [0, 16, 32, 48])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_the_choice(M, N, K, r):
    if torch.cuda.get_device_properties(0).multi_processor_count != 148:
        pytest.skip("the borders are those of 148 SMs")
    args = layer(M, N, K, r)
    ws = torch.empty(lynx.lynx_workspace_bytes(M, N, K, r), dtype=torch.uint8, device="cuda")
    for skip in (False, True) if r else (False,):
        ws.view(torch.int32).fill_(POISON)
        lynx.lynx_linear(*args, skip_sparsify=skip, workspace=ws)
        assert lynx.lynx_check_error() == (lynx.LYNX_OK, 0)
        pairs = bench.uses_pair_gemm(M, N, K, sparse=not skip, r=r)
        words = state_words(ws, M)
        assert torch.all(words != POISON) if pairs else torch.all(words == POISON), (skip, pairs, words)


def test_sparse_layers_of_a_long_k_are_the_pairs():
    """They are faster there than the 1-CTA kernel behind another that joins the partials."""
    for M, N, K, r in ((1000, 2304, 2048, 0), (1000, 2304, 2048, 16), (1000, 1504, 1792, 32), (2300, 1000, 1664, 0)):
        assert bench.uses_pair_gemm(M, N, K, r=r)
        ws = torch.full((lynx.lynx_workspace_bytes(M, N, K, r),), 0x5A, dtype=torch.uint8, device="cuda")
        lynx.lynx_linear(*layer(M, N, K, r), workspace=ws)
        assert torch.all(state_words(ws, M) != POISON), (M, N, K, r)
    assert lynx.lynx_check_error() == (lynx.LYNX_OK, 0)
