"""The scale of a packed group, pinned by rational arithmetic (CPU): the float32 quotient of
the group's range by 7 or 15, rounded to bf16."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import norm_w4 as o


def near_ties(div, binades=range(-9, -1)):
    """float32 ranges whose quotient by div lies at or next to the middle of two bf16 values,
    and whose bf16 scale another route (times the rounded 1 / div) moves by a step."""
    mid = np.concatenate([np.float32(2.0) ** e * (1 + (2 * np.arange(128) + 1) / np.float32(256)) for e in binades])
    r = (mid * div).astype(np.float32)
    r = (r.view(np.int32)[:, None] + np.arange(-4, 5)).astype(np.int32).view(np.float32).ravel()
    r = np.unique(r)
    return r[o.to_bf16(r / np.float32(div)) != o.to_bf16(r * (np.float32(1) / np.float32(div)))]


def nearest(v, bits):
    """The Fraction v > 0 to nearest-even with `bits` significant bits."""
    e = 0
    while v >= 2:
        v, e = v / 2, e + 1
    while v < 1:
        v, e = v * 2, e - 1
    n = v * 2 ** (bits - 1)
    f = n.numerator // n.denominator
    rest = n - f
    f += rest > Fraction(1, 2) or (rest == Fraction(1, 2) and f & 1)
    return Fraction(f) * Fraction(2) ** (e - bits + 1)


@pytest.mark.parametrize("div", [7, 15])
def test_scale_is_the_rounded_quotient(div):
    r = near_ties(div)
    assert r.size >= 100
    w = np.zeros((r.size, 64), np.float32)
    w[:, 5] = r
    _, s, z = o.w4_quantize(w, 64, div == 15)
    assert (z == (0 if div == 15 else 8)).all()
    for a, b in zip(r, s[:, 0]):
        assert Fraction(float(b)) == nearest(nearest(Fraction(float(a)) / div, 24), 8)
