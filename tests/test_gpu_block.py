"""The MLP half of a block end to end: norm, layers with GELU and residual in their
epilogues, checkpoints and every gradient, against automatic differentiation in 64 bits of
the same function with the selections that the forward pass made.

Tolerances, relative to the norm of what is compared.  A bf16 rounding moves a tensor by at
most 2^-8 of its norm.  Forward, X, H and h' are rounded and T twice: 5 of them, 0.02.  dh
also goes through G, dH, dZ, dX twice and dh and reads X and H from e4m3 checkpoints, whose
dX is 0.01 of its norm off at widths of 1024 (0.005 at 4096, as 1 / sqrt(K)) each: 13 of
2^-8 and 0.02, 0.071.  An adapter's A gradient sums over checkpoint values that are off by
2^-4 at most (rms below 2^-4 / sqrt(3) = 0.036) beside the same chain: 0.11.
"""
import subprocess
import sys
from pathlib import Path

import pytest
import torch

import block_oracle as oracle
from activation_sparse_gemm_lynx_b200 import lynx
from activation_sparse_gemm_lynx_b200.block import MlpBlock

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def normal(shape, seed, std):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


def layer(N, K, r, seed, skip, bias=True):
    return {"W": normal((N, K), seed, K ** -0.5), "bias": normal((N,), seed + 1, 0.02) if bias else None,
            "A": normal((r, K), seed + 2, 0.02) if r else None, "B": normal((N, r), seed + 3, 0.02) if r else None,
            "skip": skip}


def block(K=1024, F=2048, r=64, skips=(False, False), bias=True, norm=True, **kw):
    n = ((1 + 0.2 * normal((K,), 1, 1.0).float()).to(BF), normal((K,), 2, 0.1)) if norm else (None, None)
    return MlpBlock(n, layer(F, K, r, 10, skips[0], bias), layer(K, F, r, 20, skips[1], bias), **kw)


def kept(X):
    """The positions S keeps, from the oracle's S (which is nonzero at every kept value that is not zero)."""
    x = X.double()
    top = torch.sort(x.abs().reshape(x.shape[0], -1, 4), dim=2, descending=True, stable=True).indices[..., :2]
    return torch.zeros(*x.shape[:1], x.shape[1] // 4, 4, dtype=torch.float64, device=x.device).scatter_(2, top, 1.0).view_as(x)


def reference(b, h, X, H, dout=None):
    """h' in 64 bits, with the selections at the bf16 X and H; and its gradients."""
    leaves = {"h": h.double().requires_grad_()}
    for name, t in (("weight", b.weight), ("nbias", b.bias)):
        if t is not None:
            leaves[name] = t.double().requires_grad_()
    for which, lay in (("up", b.up), ("down", b.down)):
        for k in ("bias", "A", "B"):
            if lay[k] is not None:
                leaves[which + k] = lay[k].double().requires_grad_()

    def linear(x, which, lay, at):
        m = torch.ones_like(x) if lay["skip"] else kept(at)
        s = x.abs().sum(1, keepdim=True) / (m * x.abs()).sum(1, keepdim=True)
        y = (s * m * x) @ lay["W"].double().t()
        if which + "A" in leaves:
            y = y + (x @ leaves[which + "A"].t()) @ leaves[which + "B"].t()
        return y + leaves[which + "bias"] if which + "bias" in leaves else y

    x = leaves["h"]
    d = x - x.mean(1, keepdim=True)
    x = d * ((d * d).mean(1, keepdim=True) + b.eps) ** -0.5
    if "weight" in leaves:
        x = x * leaves["weight"] + leaves["nbias"]
    out = leaves["h"] + linear(oracle.gelu(linear(x, "up", b.up, X)), "down", b.down, H)
    if dout is None:
        return out, None
    grads = torch.autograd.grad(out, list(leaves.values()), dout.double())
    return out.detach(), dict(zip(leaves, grads))


def close(got, want, tol, what):
    off = float((got.double() - want).norm() / want.norm())
    assert off <= tol, f"{what}: {off:.4f} of its norm off, {tol} allowed"


@pytest.mark.parametrize("M,kw", [(700, {}), (300, dict(skips=(False, True))), (128, dict(skips=(True, False), r=16)),
                                  (257, dict(r=0, bias=False, norm=False))])
def test_forward_and_backward(M, kw):
    b = block(checkpoint=lynx.LYNX_CKPT8_E4M3, **kw)
    h, dout = normal((M, 1024), 3, 1.0), normal((M, 1024), 4, 1e-2)
    out, saved = b.forward(h, train=True)
    dh, grads = b.backward(saved, dout)
    assert lynx.lynx_check_error() == (lynx.LYNX_OK, 0)
    X = lynx.lynx_layer_norm(h, b.weight, b.bias, eps=b.eps)
    H, _ = lynx.lynx_linear_residual(X, b.up["W"], b.up["bias"], b.up["A"], b.up["B"], skip_sparsify=b.up["skip"],
                                     act=lynx.LYNX_ACT_GELU_TANH)
    want, g = reference(b, h, X, H, dout)
    close(out, want, 0.02, "h'")
    assert torch.equal(b.forward(h), out)  # the same without what a training step keeps
    close(dh, g["h"], 0.071, "dh")
    if "weight" in g:
        close(grads["norm"][0], g["weight"], 0.071, "dweight")
        close(grads["norm"][1], g["nbias"], 0.071, "dbias")
    else:
        assert grads["norm"] == (None, None)
    for which in ("up", "down"):
        assert sorted(grads[which]) == sorted(k for k in ("bias", "A", "B") if which + k in g)
        for k, got in grads[which].items():
            close(got, g[which + k], 0.11 if k == "A" else 0.071, which + k)


def test_a_captured_training_step():
    M = 300
    b = block()
    h, dout = normal((M, 1024), 3, 1.0), normal((M, 1024), 4, 1e-2)

    def flat(out, dh, grads):
        return [out, dh, *grads["norm"], *grads["up"].values(), *grads["down"].values()]

    out, saved = b.forward(h, train=True)
    first = flat(out, *b.backward(saved, dout))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, s = b.forward(h, train=True)
        captured = flat(o, *b.backward(s, dout))
    for seed in (5, 3):
        h.copy_(normal((M, 1024), seed, 1.0))
        graph.replay()
        graph.replay()
        out, saved = b.forward(h, train=True)
        now = flat(out, *b.backward(saved, dout))
        torch.cuda.synchronize()
        for x, y in zip(captured, now):
            assert torch.equal(x, y)
    for x, y in zip(first, now):  # the last replay's inputs are the first call's
        assert torch.equal(x, y)


def test_a_block_whose_first_step_is_captured():
    """The first backward pass lays out W^T: in a capture that is the graph's alone, and eager steps before and
    after a replay, of more rows too, neither read it nor move what the graph writes to."""
    b, plain = block(K=512, F=1024), block(K=512, F=1024)
    h, dout = normal((200, 512), 3, 1.0), normal((200, 512), 4, 1e-2)
    H, dOut = normal((900, 512), 5, 1.0), normal((900, 512), 6, 1e-2)

    def step(b, h, dout):
        out, saved = b.forward(h, train=True)
        dh, grads = b.backward(saved, dout)
        return [out, dh, grads["up"]["A"], grads["down"]["B"]]

    want, more = step(plain, h, dout), step(plain, H, dOut)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(b, h, dout)
    for x, y in zip(step(b, H, dOut), more):  # before any replay
        assert torch.equal(x, y)
    hold = [torch.zeros(1 << 20, device="cuda") for _ in range(16)]  # whatever is free
    graph.replay()
    torch.cuda.synchronize()
    assert all(not t.any() for t in hold)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    for x, y in zip(step(b, H, dOut), more):
        assert torch.equal(x, y)


def test_another_stream_gives_the_same():
    b = block(K=512, F=1024)
    h, dout = normal((200, 512), 3, 1.0), normal((200, 512), 4, 1e-2)
    out, saved = b.forward(h, train=True)
    dh, _ = b.backward(saved, dout)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out2, saved2 = b.forward(h, train=True)
        dh2, _ = b.backward(saved2, dout)
    side.synchronize()
    assert torch.equal(out, out2) and torch.equal(dh, dh2)


@pytest.mark.parametrize("M", [1, 7, 32])
def test_few_tokens(M):
    b = block()
    with pytest.raises(RuntimeError):
        b.forward_few(normal((M, 1024), 3, 1.0))
    b.quantize(group=64)
    h = normal((M, 1024), 3, 1.0)
    out = b.forward_few(h)
    # the dense function with the weights that the 4 bits stand for (rounded once to bf16 here)
    plain = block(skips=(True, True))
    plain.up["W"] = lynx.lynx_w4_dequantize(*b.up["w4"])
    plain.down["W"] = lynx.lynx_w4_dequantize(*b.down["w4"])
    close(out, reference(plain, h, None, None)[0].detach(), 0.02, "h'")


def test_refusals():
    up, down = layer(2048, 1024, 16, 1, False), layer(1024, 2048, 16, 2, False)
    with pytest.raises(ValueError):
        MlpBlock((None, None), up, layer(512, 2048, 16, 2, False))
    with pytest.raises(ValueError):
        MlpBlock((None, None), layer(2056, 1024, 16, 1, False), layer(1024, 2056, 16, 2, False))
    with pytest.raises(ValueError):
        MlpBlock((None, None), up, down).forward(normal((4, 512), 1, 1.0))


FIRST = """
import torch
from activation_sparse_gemm_lynx_b200 import lynx
torch.manual_seed(1)
def r(*s):
    return torch.randn(*s, device="cuda").bfloat16()
cases = []
for M, K, N in ((40, 256, 136), (700, 1024, 4096), (9, 12288, 64)):
    cases.append((r(M, K), r(N, K), r(N), r(16, K), r(N, 16), r(M, N), r(K), r(M, K), r(M, N)))
def step():
    out = []
    for X, W, bias, A, B, R, w, dX, dY in cases:
        Y, mean, rstd = lynx.lynx_layer_norm(X, w, want_stats=True)
        P, Z = lynx.lynx_linear_residual(Y, W, bias, A, B, R=R, act=lynx.LYNX_ACT_GELU_TANH, want_Z=True)
        D, _ = lynx.lynx_linear_residual(Y, W, bias, R=R, skip_sparsify=True)
        dZ, db = lynx.lynx_act_backward(dY, Z)
        _, db2 = lynx.lynx_act_backward(dY, act=lynx.LYNX_ACT_NONE)
        out += [Y, mean, rstd, P, Z, D, dZ, db, db2, *lynx.lynx_layer_norm_backward(dX, X, mean, rstd, w, dR=X)]
    return out
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
