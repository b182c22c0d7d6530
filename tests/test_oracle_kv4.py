"""Pins of oracle/kv4.py: rotation against complex numbers, codes against exact fractions, the
layout's places each used once, attention against plain sums."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import kv4 as o
from oracle.norm_w4 import to_bf16


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    g = np.random.default_rng(1)
    x = g.standard_normal((5, 3, 64))
    angle = g.uniform(0, 100, (9, 16))
    pos = np.array([0, 8, 3, 3, 5])
    y = o.rotate(x, np.cos(angle), np.sin(angle), pos, interleaved)
    i, j = (np.arange(0, 32, 2), np.arange(1, 32, 2)) if interleaved else (np.arange(16), np.arange(16, 32))
    want = (x[..., i] + 1j * x[..., j]) * np.exp(1j * angle[pos])[:, None]
    np.testing.assert_allclose(y[..., i] + 1j * y[..., j], want, atol=1e-12)
    assert np.array_equal(y[..., 32:], x[..., 32:])


@pytest.mark.parametrize("group", [32, 64, 128])
def test_codes_are_the_nearest(group):
    """By exact fractions: no other code is nearer, ties go to the even one, and a value is off by
    at most half a step and what the rounding of s to bf16 (2^-8 of it) moves code 15."""
    g = np.random.default_rng(group)
    x = to_bf16(g.standard_normal((6, 128)).astype(np.float32) * np.float32(3))
    x[1] = to_bf16(np.float32(100) + x[1] / 64)
    x[2] = 0.75
    x[3, ::2] = np.round(x[3, ::2])
    c, s, lo = o.quantize(x, group)
    for r in range(6):
        for d in range(128):
            i = d // group
            if s[r, i] == 0:
                assert c[r, d] == 0
                continue
            f = Fraction(float(np.float32(x[r, d] - lo[r, i]))) / Fraction(float(s[r, i]))
            k = int(f)
            near = k if f - k < Fraction(1, 2) or (f - k == Fraction(1, 2) and k % 2 == 0) else k + 1
            assert c[r, d] == min(near, 15)
    back = o.values(c, s, lo, group)
    step = np.repeat(s, group, -1).astype(np.float64)
    assert np.all(np.abs(back - x) <= step * (0.5 + 15 * 2.0 ** -8))
    assert np.all(o.values(c, s, lo, group).reshape(6, -1, group).min(-1) == lo)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_every_place_once(D):
    k = {tuple(int(a) for a in o.k_place(D, d)) for d in range(D)}
    assert k == {(b, up) for b in range(D // 2) for up in (0, 4)}
    v = {tuple(int(a) for a in o.v_place(D, d, t)) for d in range(D) for t in range(4)}
    assert v == {(b, up) for b in range(2 * D) for up in (0, 4)}
    # a token's bytes are its own
    assert all(o.v_place(D, d, t)[0] % 4 == t % 4 for d in range(D) for t in range(8))


def test_write_then_read():
    g = np.random.default_rng(4)
    H, D, S, group = 2, 64, 32, 32
    cache = (np.zeros((3, H, S, D // 2), np.uint8), np.zeros((3, H, 2, S, 2), np.float32),
             np.zeros((3, H, S // 4, 2 * D), np.uint8), np.zeros((3, H, 2, S, 2), np.float32))
    slots = [5, 95, 4, 33]
    x = to_bf16(g.standard_normal((2, 4, H, D)).astype(np.float32))
    parts = [o.quantize(a, group) for a in x]
    for t, slot in enumerate(slots):
        for h in range(H):
            o.write(cache, slot, h, *(a[t, h] for a in parts[0]), *(a[t, h] for a in parts[1]))
    for got, want in zip(o.read(cache, slots), parts):
        for a, b in zip(got, want):
            assert np.array_equal(a, b)


@pytest.mark.parametrize("window", [0, 1, 3])
def test_attention_by_plain_sums(window):
    g = np.random.default_rng(5)
    n, L = 6, 4  # the first two queries stand before the first key
    q, k, v = g.standard_normal((n, 4, 8)), g.standard_normal((L, 2, 8)), g.standard_normal((L, 2, 8))
    y, lse = o.attention(q, k, v, 0.3, window)
    for j in range(n):
        for i in range(4):
            at = L - n + j
            seen = [t for t in range(L) if t <= at and (not window or t > at - window)]
            w = [np.exp(0.3 * sum(q[j, i] * k[t, i // 2])) for t in seen]
            if not seen:
                assert np.all(y[j, i] == 0) and lse[j, i] == -np.inf
                continue
            np.testing.assert_allclose(y[j, i], sum(a * v[t, i // 2] for a, t in zip(w, seen)) / sum(w), rtol=1e-12)
            np.testing.assert_allclose(lse[j, i], np.log(sum(w)), rtol=1e-12, atol=1e-14)
