"""The oracle's activations and slopes against the definitions in 150 decimal
digits (1 + tanh loses 62 of them at -12), far into both tails."""
from decimal import Decimal, getcontext

import numpy as np
import pytest

from oracle import mxfp4 as mx


def exact(g, kind):
    getcontext().prec = 150
    g = Decimal(g)
    if kind == "silu":
        s, dw = 1 / (1 + (-g).exp()), Decimal(1)
    else:
        c, b = (2 / Decimal("3.14159265358979323846264338327950288419716939937511")).sqrt(), Decimal("0.044715")
        e = (2 * c * (g + b * g ** 3)).exp()
        t = (e - 1) / (e + 1)                                    # tanh
        s, dw = (1 + t) / 2, 2 * c * (1 + 3 * b * g * g)
    return g * s, s + g * s * (1 - s) * dw


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_values_and_slopes_in_both_tails(kind):
    # w's roundings, in units of 2^-53: the constant 2 sqrt(2 / pi) 2, the cubic term
    # (constant 1, cube 2, product 1), the sum 1, the product 1: 8 of |w| at most,
    # which e^w turns into relative ones; 8 more for the exponential, the quotient
    # and the products.  The slope's two terms cancel near its zero: relative to
    # their size
    for g in (-12.0, -9.75, -8.5, -7.0625, -5.5, -3.0, -1.25, -0.75, -1e-3, 0.0, 1e-3, 0.5, 2.0, 6.5, 11.0):
        a, da = exact(g, kind)
        w = abs(g) if kind == "silu" else 2 * 0.8 * (abs(g) + 0.045 * abs(g) ** 3)
        unit = (8 * w + 8) * 2.0 ** -53
        va, vda = mx.act(np.array([g]), kind)
        assert abs(Decimal(float(va[0])) - a) <= Decimal(unit) * abs(a)
        s = abs(a) / Decimal(abs(g)) if g else Decimal(1)
        dw = 1 if kind == "silu" else 1.6 * (1 + 0.135 * g * g)
        # (1 - s rounds by 2^-53 where s is near 1: that much of g dw besides)
        size = s * Decimal(1 + abs(g) * dw)
        assert abs(Decimal(float(vda[0])) - da) <= 4 * Decimal(unit) * size
