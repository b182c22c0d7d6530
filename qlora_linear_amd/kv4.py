"""A paged cache of keys and values in 4 bits (C ABI in include/kv4.h): new tokens written
to it with the position rotation on the way, rows read back, and the attention over it.

    cache = kv4_cache(n_pages, n_kv, head_dim, page_size=32, group=64)     # once a layer
    q, k, v = w4_matvec_multi(x, ...)                                      # a token a row
    q = kv4_append(q, k, v, cache, slots, cos=cos, sin=sin, positions=positions)
    y = kv4_attention(q, cache, block_table, lens)                         # one query a sequence
    y = kv4_attention(q, cache, block_table, lens, cu_q=cu_q, max_q=n)     # up to n of each
    k, v = kv4_read(cache, slots)

A cache is a tuple of four tensors, (k_codes, k_scales, v_codes, v_scales), whose shapes hold
its sizes. Like the rest of the binding these functions only check and marshal their arguments,
allocate the outputs and call the C entry point of the same name on the current stream of the
tensors' device; they synchronize nothing and may be captured into a graph. kv4_append
writes the cache in place: calls on one cache from several streams are ordered by the caller.
"""
from __future__ import annotations

import ctypes
import functools
from array import array

import torch

from . import LN_BF16, LN_F32, _SIGS, _workspace, library
from .norm_w4 import _at, _call, _code, _workspace_on

__all__ = ["kv4_cache", "kv4_append", "kv4_read", "kv4_attention", "kv4_attention_workspace_bytes", "KV4_SYMBOLS"]

_p, _i, _i64, _i32, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
_KV4_SIGS = {
    "kv4_append": (_i, [_i64, _i32, _i, _p, _i64, _p, _i64, _p, _i64, _p, _p, _i64, _i32, _i32, _p, _p, _p, _p, _p]),
    "kv4_read": (_i, [_i64, _p, _p, _i, _p, _p, _p]),
    "kv4_attention": (_i, [_i64, _i64, _i32, _p, _i64, _p, _i32, _p, _p, _i64, _i32, _f, _p, _p, _p, _p,
                           ctypes.c_size_t, _p]),
    "kv4_attention_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i32, _i32, _i32, _i32, _i64, _i32]),
}
_SIGS.update(_KV4_SIGS)
KV4_SYMBOLS = tuple(_KV4_SIGS)

_PLAIN = {torch.float32: LN_F32, torch.bfloat16: LN_BF16}
_GROUPS, _DIMS = (32, 64, 128), (64, 128, 256)
_MAX_PAGE, _MAX_HEADS = 4096, 1024
_MOST = 2 ** 31 - 1  # ctypes takes larger ones modulo 2^32


def kv4_cache(n_pages: int, n_kv: int, head_dim: int, page_size: int = 32, group: int = 64, device="cuda"):
    """(k_codes, k_scales, v_codes, v_scales) of an empty cache (all zeros) of n_pages pages of
    page_size tokens (a multiple of 32 up to 4096), n_kv heads of head_dim (64, 128 or 256) values and a
    step and a least value to `group` of them (32, 64 or 128)."""
    if head_dim not in _DIMS:
        raise ValueError(f"head_dim must be 64, 128 or 256, got {head_dim}")
    if group not in _GROUPS or head_dim % group:
        raise ValueError(f"group must be 32, 64 or 128 and divide head_dim {head_dim}, got {group}")
    if page_size < 32 or page_size % 32 or page_size > _MAX_PAGE:
        raise ValueError(f"page_size must be a multiple of 32 up to {_MAX_PAGE}, got {page_size}")
    if n_pages < 1 or not 1 <= n_kv <= _MAX_HEADS:
        raise ValueError(f"n_pages must be at least 1 and n_kv 1 to {_MAX_HEADS}, got {n_pages} and {n_kv}")
    if n_pages > _MOST or n_pages * page_size >= 1 << 40:
        raise ValueError(f"n_pages must be below 2^31 and n_pages page_size below 2^40, got {n_pages} and {page_size}")

    def tensors(*codes):
        return (torch.zeros(n_pages, n_kv, *codes, dtype=torch.uint8, device=device),
                torch.zeros(n_pages, n_kv, head_dim // group, page_size, 2, dtype=torch.bfloat16, device=device))

    return (*tensors(page_size, head_dim // 2), *tensors(page_size // 4, 2 * head_dim))


# One decoded token is a few microseconds of GPU time, so the checks below are written to
# cost little where they pass: one conjunction, and the reason worked out only on failure.

def _cache(cache):
    """(device index, n_kv, head_dim, page_size, ln_kv4_cache as an array) of a cache."""
    try:
        kc, ks, vc, vs = cache
        pages, n_kv, page, half = kc.shape
        d, groups, dev = 2 * half, ks.shape[2], kc.get_device()
        if dev >= 0 and d in _DIMS and groups * (d // groups) == d and d // groups in _GROUPS and page % 32 == 0 and \
                ks.shape == vs.shape == (pages, n_kv, groups, page, 2) and vc.shape == (pages, n_kv, page // 4, 2 * d) and \
                kc.dtype is vc.dtype is torch.uint8 and ks.dtype is vs.dtype is torch.bfloat16 and \
                ks.get_device() == vc.get_device() == vs.get_device() == dev and \
                kc.is_contiguous() and ks.is_contiguous() and vc.is_contiguous() and vs.is_contiguous():
            return dev, n_kv, d, page, array("q", (pages, page | n_kv << 32, d | d // groups << 32, kc.data_ptr(),
                                                   ks.data_ptr(), vc.data_ptr(), vs.data_ptr()))
    except (AttributeError, TypeError, ValueError, ZeroDivisionError, IndexError):
        pass  # something else than four such tensors: refused below
    if not isinstance(cache, (tuple, list)) or len(cache) != 4 or not all(isinstance(t, torch.Tensor) for t in cache):
        raise ValueError("cache must be the four tensors (k_codes, k_scales, v_codes, v_scales) of kv4_cache")
    if not all(t.is_cuda for t in cache) or len({t.get_device() for t in cache}) != 1:
        raise ValueError("cache must lie on one GPU")
    if not all(t.is_contiguous() for t in cache):
        raise ValueError("the cache's tensors must be contiguous")
    raise ValueError("cache does not have the shapes and dtypes of kv4_cache: " +
                     ", ".join(f"{t.dtype} {tuple(t.shape)}" for t in cache))


def _rows(t, name, dev, dtype, head_dim, heads=None, T=None):
    """(address, elements from row to row, T, heads) of rows [T, heads, head_dim] or
    [T, heads head_dim], which may be parts of a wider matrix's rows."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise ValueError(f"{name} must be a tensor on GPU {dev}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        n, ok = shape[1], shape[2] == head_dim and stride[2] == 1 and (shape[1] == 1 or stride[1] == head_dim)
    elif len(shape) == 2:
        n, ok = shape[1] // head_dim, shape[1] % head_dim == 0 and (stride[1] == 1 or shape[1] == 1)
    else:
        n, ok = 0, False
    if not ok or n < 1 or heads not in (None, n) or T not in (None, shape[0]):
        want = f"{'T' if T is None else T}, {'heads' if heads is None else heads}"
        raise ValueError(f"{name} must be [{want}, {head_dim}] with contiguous rows (or the last two as one), got "
                         f"{tuple(shape)} with strides {stride}")
    return t.data_ptr(), stride[0] if shape[0] > 1 else n * head_dim, shape[0], n


def _list(t, name, dev, dtype, shape):
    """The address of a list of whole numbers, and the tensor that holds it: part of a longer
    one (slots[3:5]) may start anywhere, the C entry points take 16-byte boundaries, so such
    a part is copied."""
    at = _at(t, name, dev, dtype, shape)
    if at & 15:
        t = t.clone()
        at = t.data_ptr()
    return at, t


def kv4_append(q, k, v, cache, slots, *, cos=None, sin=None, positions=None, interleaved: bool = False):
    """q rotated, as bf16 of q's shape; k rotated and v are written to the cache at `slots`.
    q [T, n_q, head_dim] (or None: only keys and values, returns None), k and v [T, n_kv, head_dim], float32 or
    bf16, all of one dtype; the last two dimensions may be one, and rows may be parts of a wider
    matrix's (a fused projection's output). slots int64 [T]: page * page_size + token; a negative
    one leaves its token out, and of tokens with the same slot the last is kept.
    cos, sin float32 [n_pos, rot_dim / 2] and positions int64 [T] (rows of them): the first rot_dim (a
    multiple of 16) elements of every head of q and k are rotated, in pairs (i, i + rot_dim / 2), or (2 i, 2 i + 1) if
    interleaved; without them nothing is. A position outside the tables leaves its token out
    and gives zeros in q."""
    dev, n_kv, d, _, c = _cache(cache)
    if not isinstance(k, torch.Tensor):
        raise ValueError("k must be a GPU tensor")
    kind = _code(_PLAIN, k.dtype, "k")
    kp, ks, T, _ = _rows(k, "k", dev, k.dtype, d, n_kv)
    vp, vs, _, _ = _rows(v, "v", dev, k.dtype, d, n_kv, T)
    sp, slots = _list(slots, "slots", dev, torch.int64, (T,))
    if (cos is None) != (sin is None) or (cos is None) != (positions is None):
        raise ValueError("cos, sin and positions go together")
    rot = n_pos = 0
    cp = np_ = pp = None
    if cos is not None:
        if not isinstance(cos, torch.Tensor) or cos.dim() != 2:
            raise ValueError("cos must be a GPU tensor [n_pos, rot_dim / 2]")
        n_pos, rot = cos.shape[0], 2 * cos.shape[1]
        if not rot or rot % 16 or rot > d:
            raise ValueError(f"cos must have a multiple of 8 columns, at most head_dim / 2, got {rot // 2}")
        cp, np_ = _at(cos, "cos", dev, torch.float32, (n_pos, rot // 2)), _at(sin, "sin", dev, torch.float32, (n_pos, rot // 2))
        pp, positions = _list(positions, "positions", dev, torch.int64, (T,))
    qp, qs, n_q, op, out = None, 0, 0, None, None
    if q is not None:
        qp, qs, _, n_q = _rows(q, "q", dev, k.dtype, d, None, T)
        out = q.new_empty(q.shape, dtype=torch.bfloat16)
        op = out.data_ptr()
    _call("kv4_append", dev, T, n_q, kind, qp, qs, kp, ks, vp, vs, cp, np_, n_pos, rot, int(interleaved), pp, sp, op,
          c.buffer_info()[0])
    return out


def kv4_read(cache, slots, dtype=torch.bfloat16):
    """(k, v) [T, n_kv, head_dim] in dtype (bf16 or float32): the cache's rows at slots int64 [T], zeros for
    one that is out of range."""
    dev, n_kv, d, _, c = _cache(cache)
    kind = _code(_PLAIN, dtype, "dtype")
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a GPU tensor [T]")
    T = slots.shape[0]
    sp, slots = _list(slots, "slots", dev, torch.int64, (T,))
    k, v = (torch.empty((T, n_kv, d), dtype=dtype, device=slots.device) for _ in range(2))
    _call("kv4_read", dev, T, sp, c.buffer_info()[0], kind, k.data_ptr(), v.data_ptr())
    return k, v


@functools.lru_cache(maxsize=256)  # (a pure function of sizes, which a decode loop repeats)
def kv4_attention_workspace_bytes(T: int, B: int, n_q: int, n_kv: int, head_dim: int, max_q: int, max_pages: int,
                                  page_size: int) -> int:
    return int(library().kv4_attention_workspace_bytes(T, B, n_q, n_kv, head_dim, max_q, max_pages, page_size))


def kv4_attention(q, cache, block_table, lens, *, cu_q=None, max_q: int | None = None, scale: float | None = None,
                  window: int = 0, return_lse: bool = False, out=None, workspace: torch.Tensor | None = None):
    """y, of q's shape, or (y, lse float32 [T, n_q]): attention of B sequences over the cache.
    q bf16 [T, n_q, head_dim] (rotated, as kv4_append returns it; rows may be parts of a wider
    matrix's), block_table int32 [B, max_pages], lens int32 [B], the keys of each sequence with its new tokens
    among them. cu_q None: a query a sequence (T = B). cu_q int32 [B + 1]: rows
    cu_q[b] .. cu_q[b + 1] - 1 are sequence b's last tokens, each of which sees the keys up to
    its own, of them the last `window` if that is not 0; max_q, if given, is at least the most
    rows of a sequence (rows past it are not written) and saves a launch where it is small. Rows
    of no sequence are left as they were, so give `out` where that matters. scale: head_dim ** -0.5 by default. A
    workspace of kv4_attention_workspace_bytes (with max_q 1 without cu_q, 0 where not given) is allocated where
    none is given."""
    dev, n_kv, d, page, c = _cache(cache)
    qp, stride, T, n_q = _rows(q, "q", dev, torch.bfloat16, d)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2 or not block_table.shape[1]:
        raise ValueError("block_table must be a GPU tensor [B, max_pages]")
    B, pages = block_table.shape
    tp, block_table = _list(block_table, "block_table", dev, torch.int32, (B, pages))
    lp, lens = _list(lens, "lens", dev, torch.int32, (B,))
    if cu_q is None:
        if T != B:
            raise ValueError(f"q has {T} rows for {B} sequences: give cu_q")
        up, bound = None, 1
    else:
        up, cu_q = _list(cu_q, "cu_q", dev, torch.int32, (B + 1,))
        bound = 0 if max_q is None else max_q
        if max_q is not None and max_q < 1:
            raise ValueError(f"max_q must be at least 1, got {max_q}")
    if window > _MOST or bound > _MOST or window < -_MOST:
        raise ValueError(f"window and max_q must be below 2^31, got {window} and {max_q}")
    if out is None:
        out = q.new_empty(q.shape)
        yp = out.data_ptr()
    else:
        yp = _at(out, "out", dev, torch.bfloat16, q.shape)
    lse = q.new_empty((T, n_q), dtype=torch.float32) if return_lse else None
    if workspace is None:
        workspace = _workspace(kv4_attention_workspace_bytes(T, B, n_q, n_kv, d, bound, pages, page), None, q.device)
    else:
        _workspace_on(dev, workspace)
    _call("kv4_attention", dev, T, B, n_q, qp, stride, up, bound, lp, tp, pages, window,
          d ** -0.5 if scale is None else scale, c.buffer_info()[0], yp, None if lse is None else lse.data_ptr(),
          None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel())
    return (out, lse) if return_lse else out
