"""Pins of the norm / packed-weight oracle (CPU): gradients against differences, codes
against brute force, the tile layout against its closed form."""
import numpy as np
import pytest

from oracle import norm_w4 as o


def test_rmsnorm_grad_against_differences():
    g = np.random.default_rng(1)
    T, d, eps = 3, 7, 1e-3
    h, w, dy, dh = g.normal(size=(T, d)), g.normal(size=d), g.normal(size=(T, d)), g.normal(size=(T, d))

    def loss(h, w):
        return (o.rmsnorm(h, w, eps)[0] * dy).sum() + (h * dh).sum()

    dx, dw = o.rmsnorm_grad(dy, h, w, o.rmsnorm(h, w, eps)[1], dh)
    step = 1e-6
    for t in range(T):
        for j in range(d):
            e = np.zeros_like(h)
            e[t, j] = step
            assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * step) - dx[t, j]) < 1e-7
    for j in range(d):
        e = np.zeros_like(w)
        e[j] = step
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * step) - dw[j]) < 1e-7


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_rows_round_to_nearest(fmt):
    g = np.random.default_rng(2)
    y = g.normal(size=(4, 33))
    y[2] = 0
    q, scale = o.quantize_rows(y, fmt)
    assert scale[2] == 0 and not q[2].any()
    levels = np.arange(-127, 128.0) if fmt == "i8" else np.array([v for v in o.e4m3_values() if v == v])
    for t in (0, 1, 3):
        v = y[t] / scale[t]
        best = np.abs(levels[None] - v[:, None]).min(1)
        assert np.all(np.abs(q[t] - v) <= best + 1e-5)
        assert np.abs(q[t]).max() == o.TOP[fmt]


@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_codes_are_nearest(group, zero_points):
    g = np.random.default_rng(3)
    w = (g.normal(size=(5, 256)) * 0.02).astype(np.float32)
    w[1, :group] = 0
    codes, s, z = o.w4_quantize(w, group, zero_points)
    rep = lambda a: np.repeat(a.astype(np.float64), group, axis=1)  # noqa: E731
    values = (np.arange(16)[None, None] - rep(z)[..., None]) * rep(s)[..., None]
    err = np.abs(o.w4_values(codes, s, z, group) - w)
    assert np.all(err <= np.abs(values - w[..., None]).min(2) + 1e-6 * np.abs(w))
    assert codes.max() <= 15 and (codes[1, :group] == z[1, 0]).all()
    if zero_points:
        assert z[1, 0] == 0
    # the largest error is half a step, or what the clamp at the scale's rounding adds
    assert np.all(err <= rep(s) * (0.5 + 15 * 2.0 ** -8))


def test_tile_layout_closed_form():
    N, K = 19, 192
    codes = np.random.default_rng(4).integers(0, 16, size=(N, K)).astype(np.uint8)
    s = np.arange(N * 3, dtype=np.float32).reshape(N, 3)
    packed, ps, _ = o.w4_pack(codes, s, s.astype(np.uint8))
    assert packed.shape == (2, 2, 1024) and ps.shape == (2, 3, 16)
    for n, k in [(0, 0), (3, 5), (15, 127), (16, 128), (18, 191), (7, 100)]:
        t, j = n % 16, k % 128
        byte = packed[n // 16, k // 128].reshape(4, 16, 4, 4)[j % 32 // 8, t, j // 32, j % 4]
        assert (byte >> (4 if j % 8 >= 4 else 0)) & 15 == codes[n, k]
        assert ps[n // 16, k // 64, n % 16] == s[n, k // 64]
    assert not packed[1].reshape(2, 4, 16, 16)[:, :, 3:].any()       # rows past d_out
    assert not packed[:, 1].reshape(2, 4, 16, 4, 4)[..., 2:, :].any()  # columns past d_in
