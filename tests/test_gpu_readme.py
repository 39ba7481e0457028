"""README.md's training sample, run as it stands there."""
from pathlib import Path

import pytest
import torch

import block_oracle as oracle
from activation_sparse_gemm_lynx_b200 import lynx

pytestmark = pytest.mark.gpu

README = Path(__file__).resolve().parent.parent / "README.md"


def normal(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def test_the_norm_and_the_residual_stream():
    """What the sample's backward calls take is what its forward calls saw: with h overwritten in between, dh
    and dweight would be those of no function."""
    text = README.read_text()
    sample = text[text.index("# the residual stream and the norm around it"):]
    sample = sample[:sample.index("\n\n")]
    M, K, r = 300, 512, 16  # one width throughout
    names = {"lynx": lynx, "h": normal((M, K), 1), "weight": normal((K,), 2), "shift": normal((K,), 3),
             "W": normal((K, K), 4, K ** -0.5), "bias": normal((K,), 5), "A": normal((r, K), 6, 0.02),
             "B": normal((K, r), 7, 0.02), "Wd": normal((K, K), 8, K ** -0.5), "bd": normal((K,), 9),
             "Ad": normal((r, K), 10, 0.02), "Bd": normal((K, r), 11, 0.02), "dH": normal((M, K), 12),
             "dX": normal((M, K), 13), "dout": normal((M, K), 14)}
    h = names["h"].clone()
    exec(compile(sample, str(README), "exec"), names)
    mean = h.float().double().mean(1)
    rstd = ((h.double() - mean[:, None]).square().mean(1) + 1e-6) ** -0.5
    want = oracle.layer_norm_backward(names["dX"], h, mean, rstd, names["weight"], names["dout"])
    # the sample's own statistics are in fp32: 2^-22 of xh more, far below a bf16 rounding
    for got, name in (("dh", "dX"), ("dweight", "dweight")):
        value, tol = want[name]
        oracle.check(names[got], (value, tol + 2.0 ** -20 * value.abs().max()), got)
    value, tol = oracle.act_backward(names["dH"], names["Z"])["dZ"]
    oracle.check(names["dZ"], (value, tol), "dZ")
    # and out is h + the second layer, with h as it was
    y = oracle.linear_residual(names["H"], names["Wd"], names["bd"], names["Ad"], names["Bd"], h, False, False)["Y"]
    oracle.check(names.get("out", names["h"]), y, "out")
