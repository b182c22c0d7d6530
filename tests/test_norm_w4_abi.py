"""C-ABI and binding checks of the norm and the packed 4-bit weight that need no GPU:
exports, and every refusal (made on the host before any HIP call)."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, ESHAPE, EALIGN, EWORKSPACE, EALIAS = 0, -1, -2, -3, -5, -6
F32, BF16, E4M3, I8 = 0, 1, 2, 3
P = 1 << 40  # plausible device-like addresses, never dereferenced


def at(i):
    return P + (i << 32)


@pytest.fixture(scope="module")
def lib():
    import qlora_linear_amd as q
    if not os.path.exists(q.library_path):
        from qlora_linear_amd import build
        build.build()
    return q.library()


def test_header_and_exports(lib):
    import qlora_linear_amd as q
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "norm_w4.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*[a-z_0-9]+\s+([a-z_0-9]+)\s*\(", text, flags=re.M)))
    assert names == sorted(q.NORM_W4_SYMBOLS)
    for n in names:
        assert hasattr(lib, n) and (n in q.__all__)


def fwd(lib, T=4, d=64, dtype=BF16, eps=1e-5, x=at(0), res=None, w=at(1), h=None, y=at(2), rstd=at(3)):
    return lib.rmsnorm_fwd(T, d, dtype, eps, x, res, w, h, y, rstd, None)


def test_rmsnorm_fwd_refusals(lib):
    assert fwd(lib, x=None) == fwd(lib, w=None) == fwd(lib, y=None) == EINVAL
    assert fwd(lib, T=-1) == fwd(lib, d=0) == fwd(lib, dtype=E4M3) == fwd(lib, dtype=7) == EINVAL
    assert fwd(lib, eps=0.0) == fwd(lib, eps=-1e-5) == EINVAL
    assert fwd(lib, eps=float("nan")) == fwd(lib, eps=float("inf")) == EINVAL
    assert fwd(lib, res=at(4)) == fwd(lib, h=at(4)) == EINVAL  # residual and h go together
    assert fwd(lib, d=(1 << 20) + 1) == fwd(lib, T=1 << 31) == ESHAPE
    assert fwd(lib, x=P + 8) == fwd(lib, rstd=at(3) + 4) == EALIGN
    assert fwd(lib, y=P) == fwd(lib, rstd=at(2)) == fwd(lib, y=at(1)) == EALIAS
    assert fwd(lib, res=at(4), h=P) == fwd(lib, res=at(4), h=at(4)) == EALIAS
    assert fwd(lib, T=0, x=None, y=None, rstd=None) == OK
    assert fwd(lib, T=0, d=0) == EINVAL


def quant(lib, T=4, d=64, dtype=BF16, x=at(0), res=None, w=at(1), h=None, qt=E4M3, q=at(2), s=at(3)):
    return lib.rmsnorm_fwd_quant(T, d, dtype, 1e-5, x, res, w, h, qt, q, s, None)


def test_rmsnorm_fwd_quant_refusals(lib):
    assert quant(lib, qt=BF16) == quant(lib, qt=F32) == quant(lib, qt=9) == quant(lib, s=None) == EINVAL
    assert quant(lib, q=None) == quant(lib, dtype=I8) == EINVAL
    assert quant(lib, q=at(2) + 8) == quant(lib, s=at(3) + 4) == EALIGN
    assert quant(lib, q=P) == quant(lib, s=at(2) + 128) == EALIAS
    assert quant(lib, T=0, x=None, q=None, s=None) == OK


def bwd(lib, T=4, d=64, dtype=BF16, dy=at(0), dh=None, h=at(1), w=at(2), rstd=at(3), dx=at(4), dw=None, ws=at(6),
        nb=None):
    if nb is None:
        nb = lib.rmsnorm_bwd_workspace_bytes(max(T, 0), d)
    return lib.rmsnorm_bwd(T, d, dtype, dy, dh, h, w, rstd, dx, dw, ws, ctypes.c_size_t(nb), None)


def test_rmsnorm_bwd_refusals(lib):
    for k in ("dy", "h", "w", "rstd", "dx"):
        assert bwd(lib, **{k: None}) == EINVAL
    assert bwd(lib, T=-1) == bwd(lib, dtype=I8) == bwd(lib, d=0) == EINVAL
    assert bwd(lib, dx=at(4) + 2) == bwd(lib, dw=at(5) + 2) == bwd(lib, dh=at(7) + 2) == EALIGN
    assert bwd(lib, dx=P) == bwd(lib, dh=at(7), dx=at(7)) == bwd(lib, dx=at(3)) == EALIAS
    assert bwd(lib, T=0, dy=None, h=None, rstd=None, dx=None) == OK
    assert lib.rmsnorm_bwd_workspace_bytes(0, 64) == 0
    assert lib.rmsnorm_bwd_workspace_bytes(8, 0) == 0
    need = lib.rmsnorm_bwd_workspace_bytes(4096, 4096)
    if need:
        assert need % 256 == 0
        assert bwd(lib, T=4096, d=4096, dw=at(5), ws=None) == EWORKSPACE
        assert bwd(lib, T=4096, d=4096, dw=at(5), nb=need - 1) == EWORKSPACE
        assert bwd(lib, T=4096, d=4096, dw=at(5), ws=at(6) + 16) == EALIGN
        assert bwd(lib, T=4096, d=4096, dw=at(5), ws=at(1)) == EALIAS


def pack(lib, w=at(0), dt=BF16, N=40, K=192, g=64, c=at(1), s=at(2), z=None):
    return lib.w4_quantize(w, dt, N, K, g, c, s, z, None)


def unpack(lib, c=at(1), s=at(2), z=None, N=40, K=192, g=64, dt=BF16, out=at(0)):
    return lib.w4_dequantize(c, s, z, N, K, g, dt, out, None)


@pytest.mark.parametrize("f", [pack, unpack])
def test_packing_refusals(lib, f):
    assert f(lib, c=None) == f(lib, s=None) == f(lib, dt=E4M3) == f(lib, N=0) == f(lib, K=0) == EINVAL
    assert f(lib, g=0) == f(lib, g=16) == f(lib, g=48) == f(lib, g=256) == ESHAPE
    assert f(lib, K=100) == f(lib, K=32, g=32) == f(lib, g=128) == f(lib, K=(1 << 22) + 64) == ESHAPE
    assert f(lib, N=1 << 31) == f(lib, N=1 << 30, K=1 << 20) == f(lib, N=1 << 28, K=64) == ESHAPE
    assert f(lib, c=at(1) + 4) == f(lib, z=at(3) + 1) == EALIGN
    assert f(lib, c=at(0)) == (EALIAS)


def mv(lib, T=2, K=192, N=40, g=64, xt=BF16, x=at(0), xs=None, c=at(1), s=at(2), z=None, yt=BF16, y=at(3), ws=None, nb=0):
    return lib.w4_matvec(T, K, N, g, xt, x, xs, c, s, z, yt, y, ws, ctypes.c_size_t(nb), None)


def test_matvec_refusals(lib):
    assert mv(lib, x=None) == mv(lib, c=None) == mv(lib, s=None) == mv(lib, y=None) == EINVAL
    assert mv(lib, T=-1) == mv(lib, N=0) == mv(lib, xt=F32) == mv(lib, yt=I8) == mv(lib, yt=E4M3) == EINVAL
    assert mv(lib, g=16) == mv(lib, g=128) == mv(lib, K=200) == mv(lib, T=(1 << 21) + 1) == ESHAPE
    assert mv(lib, x=P + 8) == mv(lib, xs=at(4) + 4) == mv(lib, z=at(5) + 8) == mv(lib, y=at(3) + 2) == EALIGN
    assert mv(lib, y=P) == mv(lib, y=at(1)) == mv(lib, xs=at(3)) == EALIAS
    assert mv(lib, T=1 << 21, N=1 << 15) == ESHAPE  # outputs of one launch
    assert mv(lib, T=0, x=None, y=None) == OK


def test_matvec_workspace(lib):
    """Only where d_in is split: deep weights of few tiles, or more rows than 16 on few tiles."""
    need = lib.w4_matvec_workspace_bytes
    assert need(1, 4096, 1024) == need(16, 8192, 28672) == need(64, 5120, 32000) == need(1, 28672, 16384) == 0
    assert need(0, 28672, 1024) == need(1, 28672 + 32, 1024) == need(1, 28672, 0) == need((1 << 21) + 1, 64, 1) == 0
    # 8 chunks of 128 are 4 steps of 2: not two splits of at least 4 steps each
    assert need(20, 1024, 40) == 0
    for T, K, N in [(16, 28672, 8192), (1, 28672, 1024), (64, 4096, 4096), (20, 2048, 40)]:
        n = need(T, K, N)
        assert n > 0 and n % 256 == 0 and n >= 2 * T * N * 4
        call = dict(T=T, K=K, N=N)
        assert mv(lib, **call) == mv(lib, **call, ws=at(6), nb=n - 1) == EWORKSPACE
        assert mv(lib, **call, ws=at(6) + 16, nb=n) == EALIGN
        assert mv(lib, **call, ws=at(1), nb=n) == mv(lib, **call, ws=at(3), nb=n) == EALIAS
    two = (ctypes.c_int64 * 2)(1024, 512)
    assert lib.w4_matvec_multi_workspace_bytes(16, 28672, 2, two) == need(16, 28672, 1536) > 0
    assert lib.w4_matvec_multi_workspace_bytes(16, 28672, 0, two) == 0
    assert lib.w4_matvec_multi_workspace_bytes(16, 28672, 2, None) == 0


def test_matvec_multi_refusals(lib):
    def call(n=2, d_out=(40, 33), c=(at(1), at(2)), s=(at(3), at(4)), z=None, y=(at(5), at(6)), T=2):
        arr = lambda a: None if a is None else (ctypes.c_void_p * len(a))(*a)  # noqa: E731
        do = None if d_out is None else (ctypes.c_int64 * len(d_out))(*d_out)
        return lib.w4_matvec_multi(T, 192, n, do, 64, BF16, at(0), None, arr(c), arr(s), arr(z), BF16, arr(y), None, 0, None)

    assert call(n=0) == call(n=9) == call(d_out=None) == call(c=None) == call(y=None) == EINVAL
    assert call(c=(at(1), None)) == call(z=(at(7), None)) == call(y=(None, at(6))) == EINVAL
    assert call(d_out=(40, 0)) == EINVAL
    assert call(y=(at(5), at(5))) == call(y=(at(5), at(5) + 64)) == call(y=(at(4), at(6))) == EALIAS
    assert call(T=0) == OK


def test_binding_refuses_host_tensors():
    import qlora_linear_amd as q
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    for f in (lambda: q.rmsnorm_fwd(x, w), lambda: q.rmsnorm_fwd_quant(x, w), lambda: q.w4_quantize(x),
              lambda: q.rmsnorm_bwd(x, x, w, torch.zeros(2)), lambda: q.w4_matvec(x, x, x)):
        with pytest.raises(ValueError, match="GPU tensor"):
            f()
