"""The operators around the NF4-LoRA linear (C ABI in include/norm_w4.h): the RMS norm
with the residual's addition, its gradient and its 8-bit output, and the product with
a 4-bit group-scaled weight.

    y, h, rstd = rmsnorm_fwd(x, w, residual=res)                  # h = x + res, y = norm(h) w
    dx, dw = rmsnorm_bwd(dy, h, w, rstd, dh=dh)                   # dx: of x and of res
    q, scale, h = rmsnorm_fwd_quant(x, w, residual=res)           # 8-bit rows, one scale each
    packed = w4_quantize(lora_nf4_merge(codes, absmax, A, B, lora_alpha), group=128)
    y = w4_matvec(q, *packed, d_out=d_out, x_scale=scale, group=128)   # (codes, scales, zeros)

Like the rest of the binding these functions only check and marshal their arguments,
allocate the outputs and call the C entry point of the same name on the current stream
of the tensors' device. They make one launch or two each and may be captured into a
graph. Gradients are functions of their own, not autograd nodes. Matrices start on 16-byte
boundaries, as PyTorch allocates them (a part of the rows of one does if a row is a multiple of
16 bytes; otherwise it is refused).
"""
from __future__ import annotations

import ctypes
from array import array

import torch

from . import LN_BF16, LN_F32, LN_MAX_PROJ, LN_OK, LoraNF4Error, _SIGS, _dev, _workspace, library

__all__ = ["rmsnorm_fwd", "rmsnorm_fwd_quant", "rmsnorm_bwd", "rmsnorm_bwd_workspace_bytes", "w4_quantize",
           "w4_dequantize", "w4_matvec", "w4_matvec_multi", "w4_matvec_workspace_bytes",
           "w4_matvec_multi_workspace_bytes", "NORM_W4_SYMBOLS", "LN_E4M3", "LN_I8"]

LN_E4M3, LN_I8 = 2, 3
LN_EWORKSPACE = -5

_p, _i, _i64, _i32, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
_NORM_W4_SIGS = {
    "rmsnorm_fwd": (_i, [_i64, _i64, _i, _f, _p, _p, _p, _p, _p, _p, _p]),
    "rmsnorm_fwd_quant": (_i, [_i64, _i64, _i, _f, _p, _p, _p, _p, _i, _p, _p, _p]),
    "rmsnorm_bwd": (_i, [_i64, _i64, _i, _p, _p, _p, _p, _p, _p, _p, _p, ctypes.c_size_t, _p]),
    "rmsnorm_bwd_workspace_bytes": (ctypes.c_size_t, [_i64, _i64]),
    "w4_quantize": (_i, [_p, _i, _i64, _i64, _i32, _p, _p, _p, _p]),
    "w4_dequantize": (_i, [_p, _p, _p, _i64, _i64, _i32, _i, _p, _p]),
    "w4_matvec": (_i, [_i64, _i64, _i64, _i32, _i, _p, _p, _p, _p, _p, _i, _p, _p, ctypes.c_size_t, _p]),
    "w4_matvec_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i64]),
    "w4_matvec_multi": (_i, [_i64, _i64, _i32, _p, _i32, _i, _p, _p, _p, _p, _p, _i, _p, _p, ctypes.c_size_t, _p]),
    "w4_matvec_multi_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i32, _p]),
}
_SIGS.update(_NORM_W4_SIGS)
NORM_W4_SYMBOLS = tuple(_NORM_W4_SIGS)

_PLAIN = {torch.float32: LN_F32, torch.bfloat16: LN_BF16}
_EIGHT = {torch.float8_e4m3fn: LN_E4M3, torch.int8: LN_I8}
_X = {torch.bfloat16: LN_BF16, **_EIGHT}
_GROUPS = (32, 64, 128)


def _code(table, dtype, name):
    code = table.get(dtype)
    if code is None:
        raise ValueError(f"{name} must have one of the dtypes {[str(t) for t in table]}, got {dtype}")
    return code


# One decoded token is a few microseconds of GPU time, so the checks below are written to
# cost little where they pass: one conjunction, and the reason worked out only on failure.

def _lead(t, name, ndim):
    """The device index of the tensor that decides where a call runs."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == ndim and t.is_contiguous():
        return t.get_device()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D")
    raise ValueError(f"{name} must be contiguous")


def _at(t, name, dev, dtype, shape):
    """The address of an operand on device `dev`, of a dtype and shape."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev and \
            t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name} must be a tensor on GPU {dev}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _row_factors(t, name, dev, T):
    """The address of one float32 a row, and the tensor that holds it: part of a batch's
    (scale[3:5]) may start anywhere, the C entry points take 16-byte boundaries, so such a
    part is copied."""
    at = _at(t, name, dev, torch.float32, (T,))
    if at & 15:
        t = t.clone()
        at = t.data_ptr()
    return at, t


def _status(name, dev, args):
    """The C entry point's status, called on the current stream of device `dev` (made the
    current device for the launch, where it is not)."""
    fn = getattr(library(), name)
    if torch._C._cuda_getDevice() == dev:
        return fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    with torch.cuda.device(dev):
        return fn(*args, torch._C._cuda_getCurrentRawStream(dev))


def _call(name, dev, *args):
    st = _status(name, dev, args)
    if st != LN_OK:
        raise LoraNF4Error(name, st)


def _workspace_on(dev, workspace):
    if _dev(workspace, "workspace", torch.uint8).get_device() != dev:
        raise ValueError(f"workspace must be a tensor on GPU {dev}")
    return workspace


def _call_matvec(name, dev, args, workspace, need, x):
    """A product on the caller's workspace, or on a new one of need() bytes where it turns out
    that one is needed (most shapes take none, and asking costs as much as trying)."""
    if workspace is None:
        st = _status(name, dev, (*args, None, 0))
        if st == LN_EWORKSPACE:
            workspace = x.new_empty(need(), dtype=torch.uint8)
            st = _status(name, dev, (*args, workspace.data_ptr(), workspace.numel()))
    else:
        _workspace_on(dev, workspace)
        st = _status(name, dev, (*args, workspace.data_ptr(), workspace.numel()))
    if st != LN_OK:
        raise LoraNF4Error(name, st)


def _norm_args(x, weight, residual):
    dev = _lead(x, "x", 2)
    kind = _code(_PLAIN, x.dtype, "x")
    T, d = x.shape
    w = _at(weight, "weight", dev, x.dtype, (d,))
    return dev, kind, T, d, w, None if residual is None else _at(residual, "residual", dev, x.dtype, (T, d))


def rmsnorm_fwd(x, weight, eps: float = 1e-5, residual=None, save_rstd: bool = True):
    """(y, h, rstd): h = x + residual rounded to x's dtype (x itself without a residual),
    y = h * rstd * weight, rstd = 1 / sqrt(mean(h^2) + eps) float32 [T] (None unless
    save_rstd). x [T, d] float32 or bf16; weight [d] and residual [T, d] of the same dtype."""
    dev, kind, T, d, w, r = _norm_args(x, weight, residual)
    y = torch.empty_like(x)
    h = x if residual is None else torch.empty_like(x)
    rstd = x.new_empty(T, dtype=torch.float32) if save_rstd else None
    _call("rmsnorm_fwd", dev, T, d, kind, eps, x.data_ptr(), r, w, None if r is None else h.data_ptr(),
          y.data_ptr(), None if rstd is None else rstd.data_ptr())
    return y, h, rstd


def rmsnorm_fwd_quant(x, weight, eps: float = 1e-5, residual=None, qdtype=torch.float8_e4m3fn):
    """(q, scale, h): the norm's rows as qdtype (torch.float8_e4m3fn or torch.int8) [T, d] and
    one float32 scale a row [T], y = q * scale; h as for rmsnorm_fwd."""
    dev, kind, T, d, w, r = _norm_args(x, weight, residual)
    fmt = _code(_EIGHT, qdtype, "qdtype")
    q = torch.empty_like(x, dtype=qdtype)
    scale = x.new_empty(T, dtype=torch.float32)
    h = x if residual is None else torch.empty_like(x)
    _call("rmsnorm_fwd_quant", dev, T, d, kind, eps, x.data_ptr(), r, w, None if r is None else h.data_ptr(), fmt,
          q.data_ptr(), scale.data_ptr())
    return q, scale, h


def rmsnorm_bwd_workspace_bytes(T: int, d: int) -> int:
    return int(library().rmsnorm_bwd_workspace_bytes(T, d))


def rmsnorm_bwd(dy, h, weight, rstd, dh=None, need_dw: bool = True, workspace: torch.Tensor | None = None):
    """(dx, dw or None) of rmsnorm_fwd for the gradient dy of y and, if given, the gradient dh
    that reaches h from its other readers; dx is the gradient of x and of the residual."""
    dev = _lead(h, "h", 2)
    kind = _code(_PLAIN, h.dtype, "h")
    T, d = h.shape
    w = _at(weight, "weight", dev, h.dtype, (d,))
    g = _at(dy, "dy", dev, h.dtype, (T, d))
    r, rstd = _row_factors(rstd, "rstd", dev, T)
    e = None if dh is None else _at(dh, "dh", dev, h.dtype, (T, d))
    dx = torch.empty_like(h)
    dw = torch.empty_like(weight) if need_dw else None
    if workspace is not None:
        _workspace_on(dev, workspace)
    ws = _workspace(rmsnorm_bwd_workspace_bytes(T, d), workspace, h.device) if need_dw else None
    _call("rmsnorm_bwd", dev, T, d, kind, g, e, h.data_ptr(), w, r, dx.data_ptr(),
          None if dw is None else dw.data_ptr(), None if ws is None else ws.data_ptr(),
          0 if ws is None else ws.numel())
    return dx, dw


def w4_quantize(w, group: int = 128, zero_points: bool = False):
    """(codes, scales, zeros or None): w [d_out, d_in] float32 or bf16 packed to 4 bits with one
    bf16 scale (and zero point) per row and `group` columns (32, 64 or 128; d_in a multiple of
    64 and of group), laid out in tiles of 16 rows x 128 columns as norm_w4.h describes."""
    dev = _lead(w, "w", 2)
    kind = _code(_PLAIN, w.dtype, "w")
    N, K = w.shape
    if group not in _GROUPS:
        raise ValueError(f"group must be 32, 64 or 128, got {group}")
    nt, kt, kg = (N + 15) // 16, (K + 127) // 128, K // group
    codes = w.new_empty((nt, kt, 1024), dtype=torch.uint8)
    scales = w.new_empty((nt, kg, 16), dtype=torch.bfloat16)
    zeros = w.new_empty((nt, kg, 16), dtype=torch.uint8) if zero_points else None
    _call("w4_quantize", dev, w.data_ptr(), kind, N, K, group, codes.data_ptr(), scales.data_ptr(),
          None if zeros is None else zeros.data_ptr())
    return codes, scales, zeros


# A packed weight's tensors do not hold its width: 64 columns fill half a tile, and with groups
# of 32 (64) they have the shapes of 128 columns with groups of 64 (128).

def _columns(codes, scales, group):
    """d_in of a packed weight from its shapes, and its group size if given."""
    if not isinstance(scales, torch.Tensor) or scales.dim() != 3 or not scales.shape[1]:
        raise ValueError("scales must be [ceil(d_out / 16), d_in / group, 16]")
    full, kg = codes.shape[1] * 128, scales.shape[1]
    fits = [k for k in (full, full - 64) if k % kg == 0 and k // kg in _GROUPS and group in (None, k // kg)]
    if len(fits) != 1:
        raise ValueError(f"{codes.shape[1]} tiles and {kg} groups of a row with group {group} " +
                         ("are 64 or 128 columns: give d_in or group" if fits else "are no packed weight"))
    return fits[0]


def _packed(codes, scales, zeros, d_in, d_out, dev, index=None, want=None):
    """(d_out, group, addresses) of a packed weight whose rows are d_in wide; index: its
    place in a list, for errors; want: the group size that it must have."""
    try:
        nt, kg, rows = scales.shape
        group = d_in // kg
        n = 16 * nt if d_out is None else d_out
        if rows == 16 and group in _GROUPS and kg * group == d_in and 16 * (nt - 1) < n <= 16 * nt and \
                want in (None, group) and \
                scales.dtype is torch.bfloat16 and scales.get_device() == dev and scales.is_contiguous() and \
                codes.dtype is torch.uint8 and codes.shape == (nt, (d_in + 127) // 128, 1024) and \
                codes.get_device() == dev and codes.is_contiguous():
            if zeros is None:
                return n, group, codes.data_ptr(), scales.data_ptr(), 0
            if zeros.dtype is torch.uint8 and zeros.shape == (nt, kg, 16) and zeros.get_device() == dev and \
                    zeros.is_contiguous():
                return n, group, codes.data_ptr(), scales.data_ptr(), zeros.data_ptr()
    except (AttributeError, TypeError, ValueError, ZeroDivisionError):
        pass  # something else than such tensors: refused below
    tag = "" if index is None else f"[{index}]"
    if not isinstance(scales, torch.Tensor) or scales.dim() != 3 or scales.shape[2] != 16 or not scales.shape[1]:
        raise ValueError(f"scales{tag} must be [ceil(d_out / 16), d_in / group, 16]")
    nt, kg, _ = scales.shape
    if kg * (d_in // kg) != d_in or d_in // kg not in _GROUPS:
        raise ValueError(f"scales{tag} hold {kg} groups of a row: d_in {d_in} makes no group of 32, 64 or 128")
    if want is not None and want * kg != d_in:
        raise ValueError(f"scales{tag} hold {kg} groups of a row: {want} columns each are not d_in {d_in}")
    if d_out is not None and not 16 * (nt - 1) < d_out <= 16 * nt:
        raise ValueError(f"d_out{tag} {d_out} does not fit scales{tag} of {nt} tiles of 16 rows")
    _at(scales, f"scales{tag}", dev, torch.bfloat16, (nt, kg, 16))
    _at(codes, f"codes{tag}", dev, torch.uint8, (nt, (d_in + 127) // 128, 1024))
    _at(zeros, f"zeros{tag}", dev, torch.uint8, (nt, kg, 16))
    raise ValueError(f"packed weight{tag} not understood")


def w4_dequantize(codes, scales, zeros=None, *, d_out: int | None = None, d_in: int | None = None,
                  dtype=torch.bfloat16, group: int | None = None):
    """[d_out, d_in] float32 or bf16 values of a packed weight. Defaults: every row that the
    tiles hold, and the d_in that the shapes stand for; where they stand for 64 columns as
    well as for 128 (one tile a row with one or two groups), d_in or group has to be given."""
    dev = _lead(codes, "codes", 3)
    kind = _code(_PLAIN, dtype, "dtype")
    K = _columns(codes, scales, group) if d_in is None else d_in
    N, group, c, s, z = _packed(codes, scales, zeros, K, d_out, dev, None, group)
    out = codes.new_empty((N, K), dtype=dtype)
    _call("w4_dequantize", dev, c, s, z, N, K, group, kind, out.data_ptr())
    return out


def _x_args(x, x_scale, dtype):
    dev = _lead(x, "x", 2)
    xs, held = (None, None) if x_scale is None else _row_factors(x_scale, "x_scale", dev, x.shape[0])
    return dev, _code(_X, x.dtype, "x"), xs, held, _code(_PLAIN, dtype, "dtype")


def w4_matvec_workspace_bytes(T: int, d_in: int, d_out: int) -> int:
    return int(library().w4_matvec_workspace_bytes(T, d_in, d_out))


def w4_matvec_multi_workspace_bytes(T: int, d_in: int, d_outs) -> int:
    widths = array("q", d_outs)
    return int(library().w4_matvec_multi_workspace_bytes(T, d_in, len(widths), widths.buffer_info()[0]))


def w4_matvec(x, codes, scales, zeros=None, *, d_out: int | None = None, x_scale=None, dtype=torch.bfloat16,
              out=None, workspace: torch.Tensor | None = None, group: int | None = None):
    """y = (x_scale x) W^T [T, d_out] in dtype (float32 or bf16) for x [T, d_in] bf16, float8_e4m3fn
    or int8 and a packed weight; x_scale: float32 [T] or None. Made for up to 64 rows. A workspace is
    allocated where one is needed (w4_matvec_workspace_bytes) and none is given.
    x's width is the weight's d_in; the shapes alone cannot tell a weight of 64 columns from one
    of 128 with groups twice as large, so where that may be mixed up give the group size too: a
    weight of other groups is then refused."""
    dev, xt, xs, x_scale, yt = _x_args(x, x_scale, dtype)
    T, K = x.shape
    N, group, c, s, z = _packed(codes, scales, zeros, K, d_out, dev, None, group)
    if out is None:
        out = x.new_empty((T, N), dtype=dtype)
        y = out.data_ptr()
    else:
        y = _at(out, "out", dev, dtype, (T, N))
    _call_matvec("w4_matvec", dev, (T, K, N, group, xt, x.data_ptr(), xs, c, s, z, yt, y), workspace,
                 lambda: w4_matvec_workspace_bytes(T, K, N), x)
    return out


def w4_matvec_multi(x, codes, scales, zeros=None, *, d_out=None, x_scale=None, dtype=torch.bfloat16,
                    workspace: torch.Tensor | None = None, group: int | None = None):
    """[y_g] of several packed weights (lists, one entry per weight) that read the same x, as one
    w4_matvec each but together in one launch. zeros: None, or one entry per weight."""
    dev, xt, xs, x_scale, yt = _x_args(x, x_scale, dtype)
    T, K = x.shape
    n = len(codes)
    if not 1 <= n <= LN_MAX_PROJ or len(scales) != n or (zeros is not None and len(zeros) != n) or \
            (d_out is not None and len(d_out) != n):
        raise ValueError(f"codes, scales (zeros, d_out) must be lists of the same length, 1 to {LN_MAX_PROJ}")
    N, groups, c, s, z = zip(*(_packed(codes[g], scales[g], None if zeros is None else zeros[g], K,
                                       None if d_out is None else d_out[g], dev, g, group) for g in range(n)))
    if len(set(groups)) > 1:
        raise ValueError("all weights must share the group size")
    if not all(z) and any(z):
        raise ValueError("zeros must be given for every weight or for none")
    ys = [x.new_empty((T, w), dtype=dtype) for w in N]
    # the five arrays of the C call side by side (read during the call only)
    table = array("q", (*N, *c, *s, *z, *(y.data_ptr() for y in ys)))
    at, _ = table.buffer_info()
    _call_matvec("w4_matvec_multi", dev, (T, K, n, at, groups[0], xt, x.data_ptr(), xs, at + 8 * n, at + 16 * n,
                                          at + 24 * n if z[0] else None, yt, at + 32 * n), workspace,
                 lambda: w4_matvec_multi_workspace_bytes(T, K, N), x)
    return ys
