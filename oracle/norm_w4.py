"""RMS norm (forward, 8-bit rows, backward) and the packed 4-bit weight — oracle.

TEST INFRASTRUCTURE ONLY (see the package docstring). Plain numpy: products and sums
in float64; the steps whose rounding is part of the definition (h, the scales, the
codes of a weight) in the format that the definition rounds to.
"""
from __future__ import annotations

import numpy as np

from .dq import e4m3_encode, e4m3_values

TOP = {"e4m3": 448.0, "i8": 127.0}


def to_bf16(a) -> np.ndarray:
    """float32 values rounded to nearest-even bf16, as float32."""
    u = np.ascontiguousarray(a, dtype=np.float32).view(np.uint32)
    u = u + (((u >> np.uint32(16)) & np.uint32(1)) + np.uint32(0x7FFF))
    return (u & np.uint32(0xFFFF0000)).view(np.float32)


def rmsnorm(h, w, eps):
    """(y, rstd) in float64 of rows h and weight w."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * w, rstd


def quantize_rows(y, fmt):
    """(levels float64, scale) of 8-bit rows: y / scale rounded to the format's nearest."""
    scale = np.abs(y).max(1) / TOP[fmt]
    v = np.divide(y, scale[:, None], out=np.zeros_like(y), where=scale[:, None] > 0)
    if fmt == "i8":
        return np.rint(v), scale
    return e4m3_values()[e4m3_encode(v.astype(np.float32))].reshape(y.shape), scale


def rmsnorm_grad(dy, h, w, rstd, dh=None):
    """(dx, dw) in float64."""
    dy, h, w, r = (np.asarray(a, np.float64) for a in (dy, h, w, rstd))
    g, n = dy * w, h * r[:, None]
    dx = r[:, None] * (g - n * (g * n).mean(1, keepdims=True))
    return (dx if dh is None else dx + np.asarray(dh, np.float64)), (dy * n).sum(0)


def w4_quantize(w, group, zero_points):
    """(codes [N, K], scales float32 (bf16 values) [N, K / group], zeros [N, K / group]):
    float32 steps, each rounded to nearest-even, as the format defines them."""
    w = np.asarray(w, np.float32)
    N, K = w.shape
    g = w.reshape(N, K // group, group)
    if zero_points:
        lo, hi = np.minimum(g.min(2), 0), np.maximum(g.max(2), 0)
        s = to_bf16((hi - lo) / np.float32(15))
        z = np.divide(-lo, s, out=np.zeros_like(s), where=s > 0)
        z = np.clip(np.rint(z), 0, 15)
    else:
        s = to_bf16(np.abs(g).max(2) / np.float32(7))
        z = np.full_like(s, 8)
    v = np.divide(g, s[..., None], out=np.zeros_like(g), where=s[..., None] > 0)
    c = np.clip(np.rint(v) + z[..., None], 0, 15)
    return c.reshape(N, K).astype(np.uint8), s, z.astype(np.uint8)


def w4_values(codes, scales, zeros, group):
    """float64 [N, K] of unpacked codes."""
    rep = lambda a: np.repeat(np.asarray(a, np.float64), group, axis=1)  # noqa: E731
    return (codes.astype(np.float64) - rep(zeros)) * rep(scales)


def w4_pack(codes, scales, zeros):
    """The tile layout, element by element: (codes uint8 [nt, kt, 1024], scales, zeros [nt, groups, 16])."""
    N, K = codes.shape
    nt, kt = (N + 15) // 16, (K + 127) // 128
    out = np.zeros((nt, kt, 1024), np.uint8)
    n, k = np.meshgrid(np.arange(N), np.arange(K), indexing="ij")
    kk = k % 128
    byte = 256 * (kk % 32 // 8) + 16 * (n % 16) + 4 * (kk // 32) + kk % 4
    np.bitwise_or.at(out, (n // 16, k // 128, byte), codes << (4 * (kk % 8 // 4)).astype(np.uint8))

    def per_group(a):
        t = np.zeros((nt * 16, a.shape[1]), a.dtype)
        t[:N] = a
        return np.ascontiguousarray(t.reshape(nt, 16, -1).transpose(0, 2, 1))

    return out, per_group(scales), per_group(zeros)
