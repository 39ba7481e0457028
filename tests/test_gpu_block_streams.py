"""MlpBlock's layouts of W across streams and captures."""
import pytest
import torch

from activation_sparse_gemm_lynx_b200 import lynx
from activation_sparse_gemm_lynx_b200.block import MlpBlock

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def normal(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


def block(K=512, F=1024, r=16):
    def layer(N, K, seed):
        return {"W": normal((N, K), seed, K ** -0.5), "bias": normal((N,), seed + 1, 0.02),
                "A": normal((r, K), seed + 2, 0.02), "B": normal((N, r), seed + 3, 0.02)}

    return MlpBlock((normal((K,), 1), normal((K,), 2)), layer(F, K, 10), layer(K, F, 20))


def test_quantized_on_one_stream_and_served_on_another():
    """quantize() returns once the layout is there, whatever its stream still had to do before."""
    plain, b = block(), block()
    h = normal((5, 512), 3)
    plain.quantize(group=64)
    want = plain.forward_few(h)
    big = normal((8192, 8192), 4, 0.01)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(5):  # milliseconds before the layout's turn comes
            big @ big
        b.quantize(group=64)
    assert side.query()
    assert torch.equal(b.forward_few(h), want)
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        got = b.forward_few(h)
    other.synchronize()
    assert torch.equal(got, want)


def test_quantize_inside_a_capture_is_refused():
    """The graph's memory would hold no layout before a replay, and every eager call would read it."""
    b = block()
    h = normal((5, 512), 3)
    x = torch.zeros(8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.add_(1)
        with pytest.raises(RuntimeError, match="before the capture"):
            b.quantize()
    with pytest.raises(RuntimeError, match="quantize"):
        b.forward_few(h)
    b.quantize()
    want = b.forward_few(h)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph := torch.cuda.CUDAGraph()):
        got = b.forward_few(h)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert lynx.lynx_check_error()[0] == lynx.LYNX_OK
