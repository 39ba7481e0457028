"""Relative norm errors, beside the element bounds of adapter_oracle.py.

An element bound that adds every rounding in the worst direction grows with the
length of the sums, so that at large sizes a wrong operand can pass under it.  In the
norm the roundings add as they come: a result rounded once is off by the norm of
that rounding, which the reference itself gives.
"""
import torch

# What fp32 sums and operands of 16 bits or more add before the last rounding.  A sum of
# n products in steps of 16 loses at most 2^-23 of the running sum a step; with running
# sums up to 4 times the result and n / 16 <= 288 (n <= 4608) that is 288 * 4 * 2^-23 =
# 1.4e-4, and two operands of 16 bits are off by 2 * 2^-17 = 1.5e-5: below 2^-12 together.
SUMS = 2.0 ** -12


def rounded_once(got, ref, dim=None):
    """Asserts ||got - ref|| <= 1.1 ||bf16(ref) - ref|| + 2^-12 ||ref||, over all or along `dim`.

    1.1: the norm of n roundings that fall anywhere within half a step scatters by about
    1 / sqrt(n) of itself, and the cases have over 500 values each.  One more rounding to bf16 of an operand of
    the sum adds as much again in the other direction of the square: a factor of 1.41."""
    if dim is None:
        got, ref, dim = got.reshape(-1), ref.reshape(-1), 0
    off = (got.double() - ref).norm(dim=dim)
    most = 1.1 * (ref.bfloat16().double() - ref).norm(dim=dim) + SUMS * ref.norm(dim=dim)
    worst = float((off / most.clamp(min=2.0 ** -126)).max())
    assert worst <= 1, worst
