"""Where a row of Y may begin: on 16 bytes, whatever N and the kernel that writes it."""
import pytest
import torch

from activation_sparse_gemm_lynx_b200 import lynx

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def normal(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


# tiles of 32 to 256 columns, the last one whole, ragged and of 8 columns; N on 32 bytes and only on 16
@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 8, 64), (7, 64, 64), (37, 4096, 192), (100, 9224, 192), (300, 1536, 192), (300, 1544, 192),
                                   (1000, 2304, 192), (1000, 2296, 192), (4000, 520, 192), (5000, 4368, 64), (1300, 2064, 256)])
def test_y_on_16_bytes_and_nothing_around_it(M, N, K, skip):
    X, W, bias, R = normal((M, K), 1), normal((N, K), 2, K ** -0.5), normal((N,), 3), normal((M, N), 4)
    want = lynx.lynx_linear(X, W, bias, skip_sparsify=skip)
    assert want.data_ptr() % 256 == 0
    kw = dict(R=R, skip_sparsify=skip, act=lynx.LYNX_ACT_GELU_TANH)
    ext, Z = lynx.lynx_linear_residual(X, W, bias, want_Z=True, **kw)
    assert torch.equal(Z, want)
    for off in (0, 8, 16):  # elements: on 32 bytes, on 16 only, on 32
        room = torch.full((3, 64 + M * N + 64), 7.0, dtype=BF, device="cuda")
        at = [room[i, off + 16:off + 16 + M * N].view(M, N) for i in range(3)]
        lynx.lynx_linear(X, W, bias, skip_sparsify=skip, Y=at[0])
        lynx.lynx_linear_residual(X, W, bias, Y=at[1], Z=at[2], **kw)
        assert torch.equal(at[0], want) and torch.equal(at[1], ext) and torch.equal(at[2], Z), off
        assert torch.all(room[:, :off + 16] == 7.0) and torch.all(room[:, off + 16 + M * N:] == 7.0)
    assert lynx.lynx_check_error() == (lynx.LYNX_OK, 0)
