"""Bounds of the layers' arithmetic that are relative to what is computed, beside the worst-case ones of
tests/layer_oracle.py. Shares no code with the library."""
import math

import torch

from tests import layer_oracle as oracle

# The activations' own error, relative to their value. Float results: the fit of the normal distribution's tail
# 1.8e-8, about a rounding each (2^-24) of its eight steps (the later ones count most: together 4), of the reciprocal,
# the exponential (2 and its correction), three products, the difference from 1 and the last product: at most 16, so
# 2^-20. Results of 2 bytes: a fit of at most 5.9e-6 and the rounded argument of the exponential, at most
# 128 * 2^-24 = 7.6e-6 before it underflows: 2^-16, a thirty-second of half's half step.
RELATIVE = {4: 2.0 ** -20, 2: 2.0 ** -16}
# Exponentials below the smallest normal float are 0: at most 90 times that is lost of a value.
FLOOR = 90 * 2.0 ** -126


def value_bound(y, out):
    return RELATIVE[out.itemsize] * y.abs() + FLOOR + oracle.rounding(y, out)


def slope_parts(z, name):
    """The slope and the sum of its terms' magnitudes."""
    if name == "gelu":
        a = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        b = z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    else:
        q = torch.sigmoid(z)
        a, b = q, z * q * torch.sigmoid(-z)
    return a + b, a + b.abs()


def norm_check(got, want, terms, dtype, what, roundings=1):
    """Error in the 2-norm of a sum of `terms` products of either sign, rounded `roundings` times to `dtype`. A float
    addition is off by at most 2^-23 of the partial sum (truncation included) with no common sign, so the errors of a
    sum add up as the root of their number; a rounding is off by at most half a step of each entry."""
    got, want = got.double(), want.double()
    off = float((got - want).norm() / want.norm())
    bound = math.sqrt(terms + 8) * 2.0 ** -23 + roundings * oracle.EPS[dtype] / 2
    assert off <= bound, (what, off, bound)
