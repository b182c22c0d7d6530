"""A paged cache of keys and values in 4 bits, and attention over it — oracle.

TEST INFRASTRUCTURE ONLY (see the package docstring). Plain numpy: products and sums in
float64; the steps whose rounding is part of the definition (rotated rows, steps, codes) in
the format that the definition rounds to. Layout: element by element.
"""
from __future__ import annotations

import numpy as np

from .norm_w4 import to_bf16


def rotate(x, cos, sin, positions, interleaved):
    """float64 rows [T, H, D]: the pairs of the first 2 cos.shape[1] elements turned by their
    position's angles."""
    x = np.asarray(x, np.float64).copy()
    n = cos.shape[1]
    c, s = (np.asarray(a, np.float64)[positions][:, None] for a in (cos, sin))
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    a, b = x[..., i].copy(), x[..., j].copy()
    x[..., i], x[..., j] = a * c - b * s, b * c + a * s
    return x


def rounded(x):
    """float64 rounded to float32 and then to bf16 (as float32)."""
    return to_bf16(np.asarray(x, np.float64).astype(np.float32))


def quantize(x, group):
    """(codes [.., D] uint8, s [.., D / group], lo) of bf16 values held as float32."""
    x = np.asarray(x, np.float32)
    v = x.reshape(*x.shape[:-1], -1, group)
    lo, hi = v.min(-1), v.max(-1)
    s = to_bf16((hi - lo) / np.float32(15))
    d = (v - lo[..., None]).astype(np.float64)
    c = np.divide(d, s[..., None], out=np.zeros_like(d), where=s[..., None] > 0)
    return np.minimum(np.rint(c), 15).astype(np.uint8).reshape(x.shape), s, lo


def values(codes, s, lo, group):
    """float64 values of codes [.., D]."""
    rep = lambda a: np.repeat(np.asarray(a, np.float64), group, axis=-1)  # noqa: E731
    return codes.astype(np.float64) * rep(s) + rep(lo)


def k_place(D, d):
    """(byte of a key's row, shift of the nibble) of element d."""
    c, r = d // 32, d % 32
    return r // 8 * (D // 8) + 4 * c + r % 4, 4 * (r % 8 // 4)


def v_place(D, d, tok):
    """(byte of four tokens' values, shift) of element d of token tok."""
    c, r = d // 32, d % 32
    return r // 2 * (D // 8) + 4 * c + tok % 4, 4 * (d % 2)


def write(cache, slot, h, kc, ks, klo, vc, vs, vlo):
    """One head of one slot into cache = numpy (k_codes, k_scales, v_codes, v_scales), the
    scales as float32; codes [D], s and lo [D / group]."""
    k_codes, k_scales, v_codes, v_scales = cache
    S, D = k_codes.shape[2], kc.size
    page, tok = slot // S, slot % S
    for d in range(D):
        for tab, (byte, up), code in ((k_codes[page, h, tok], k_place(D, d), kc[d]),
                                      (v_codes[page, h, tok // 4], v_place(D, d, tok), vc[d])):
            tab[byte] = (int(tab[byte]) & (0xF0 if up == 0 else 0x0F)) | (int(code) << up)
    k_scales[page, h, :, tok, 0], k_scales[page, h, :, tok, 1] = ks, klo
    v_scales[page, h, :, tok, 0], v_scales[page, h, :, tok, 1] = vs, vlo


def read(cache, slots):
    """(k, v) parts (codes [T, H, D], s, lo [T, H, D / group]) of slots, by numpy indexing."""
    k_codes, k_scales, v_codes, v_scales = cache
    S, D = k_codes.shape[2], 2 * k_codes.shape[3]
    slots = np.asarray(slots)
    page, tok, d = slots // S, slots % S, np.arange(D)
    byte, up = k_place(D, d)
    kc = (k_codes[page, :, tok][..., byte] >> up) & 15
    byte, up = v_place(D, d[None], tok[:, None])
    quad = v_codes[page, :, tok // 4]
    vc = (np.take_along_axis(quad, np.broadcast_to(byte[:, None], (*quad.shape[:2], D)), -1) >> up[:, None]) & 15
    ks, vs = k_scales[page, :, :, tok], v_scales[page, :, :, tok]
    return (kc, ks[..., 0], ks[..., 1]), (vc, vs[..., 0], vs[..., 1])


def attention(q, k, v, scale, window=0):
    """(y [n, Hq, D], lse [n, Hq]) in float64 of n queries that stand for the last n of the L keys
    k, v [L, H, D]; rows that see no key: y 0, lse -inf."""
    n, hq, _ = q.shape
    L, h, _ = k.shape
    y, lse = np.zeros(q.shape), np.full((n, hq), -np.inf)
    for j in range(n):
        hi = L - n + j + 1
        lo = max(0, hi - window) if window else 0
        if hi <= lo:
            continue
        for i in range(hq):
            g = i // (hq // h)
            x = scale * (k[lo:hi, g] @ q[j, i])
            m = x.max()
            p = np.exp(x - m)
            y[j, i] = p @ v[lo:hi, g] / p.sum()
            lse[j, i] = m + np.log(p.sum())
    return y, lse
