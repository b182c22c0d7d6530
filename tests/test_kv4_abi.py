"""C-ABI and binding checks of the paged 4-bit cache that need no GPU: exports, and every
refusal (made on the host before any HIP call)."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, ESHAPE, EALIGN, EWORKSPACE, EALIAS = 0, -1, -2, -3, -5, -6
F32, BF16, E4M3 = 0, 1, 2
P = 1 << 40  # plausible device-like addresses, never dereferenced


def at(i):
    return P + (i << 36)


class Cache(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("n_kv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("group", ctypes.c_int32), ("kc", ctypes.c_void_p), ("ks", ctypes.c_void_p),
                ("vc", ctypes.c_void_p), ("vs", ctypes.c_void_p)]


def cache(n_pages=7, page=32, n_kv=2, d=64, group=32, kc=at(20), ks=at(21), vc=at(22), vs=at(23)):
    return ctypes.byref(Cache(n_pages, page, n_kv, d, group, kc, ks, vc, vs))


@pytest.fixture(scope="module")
def lib():
    import qlora_linear_amd as q
    if not os.path.exists(q.library_path):
        from qlora_linear_amd import build
        build.build()
    return q.library()


def test_header_and_exports(lib):
    import qlora_linear_amd as q
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "kv4.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*[a-z_0-9]+\s+([a-z_0-9]+)\s*\(", text, flags=re.M)))
    assert names == sorted(q.KV4_SYMBOLS)
    for n in names:
        assert hasattr(lib, n) and (n in q.__all__)


def append(lib, T=3, n_q=4, dt=BF16, q=at(0), qs=256, k=at(1), ks=128, v=at(2), vs=128, cos=at(3), sin=at(4), n_pos=10,
           rot=32, inter=0, pos=at(5), slots=at(6), out=at(7), c=cache()):
    return lib.kv4_append(T, n_q, dt, q, qs, k, ks, v, vs, cos, sin, n_pos, rot, inter, pos, slots, out, c, None)


def read(lib, T=3, slots=at(6), c=cache(), dt=BF16, k=at(0), v=at(1)):
    return lib.kv4_read(T, slots, c, dt, k, v, None)


def attend(lib, T=3, B=3, n_q=4, q=at(0), qs=256, cu=None, max_q=0, lens=at(1), table=at(2), pages=5, window=0, scale=0.1,
           c=cache(), y=at(3), lse=None, ws=at(5), nb=1 << 40):
    return lib.kv4_attention(T, B, n_q, q, qs, cu, max_q, lens, table, pages, window, scale, c, y, lse, ws,
                             ctypes.c_size_t(nb), None)


@pytest.mark.parametrize("f", [append, read, attend])
def test_cache_refusals(lib, f):
    assert f(lib, c=None) == EINVAL
    for name in ("kc", "ks", "vc", "vs"):
        assert f(lib, c=cache(**{name: None})) == EINVAL
        assert f(lib, c=cache(**{name: at(20) + 8})) == EALIGN
    for bad in (dict(n_pages=0), dict(n_pages=-1), dict(n_kv=0), dict(page=0), dict(d=0)):
        assert f(lib, c=cache(**bad)) == EINVAL
    for bad in (dict(page=16), dict(page=48), dict(page=4128), dict(d=32), dict(d=96), dict(d=512), dict(group=16),
                dict(group=96), dict(group=128), dict(n_kv=1025), dict(n_pages=1 << 31), dict(n_pages=1 << 30, page=1024)):
        assert f(lib, c=cache(**bad)) == ESHAPE


def test_append_refusals(lib):
    assert append(lib, T=-1) == append(lib, dt=E4M3) == append(lib, rot=-16) == append(lib, inter=2) == EINVAL
    assert append(lib, q=None) == append(lib, out=None) == append(lib, k=None) == append(lib, v=None) == EINVAL
    assert append(lib, slots=None) == append(lib, pos=None) == append(lib, n_q=0) == append(lib, n_pos=0) == EINVAL
    assert append(lib, cos=None) == append(lib, sin=None) == append(lib, rot=0) == EINVAL
    assert append(lib, rot=8) == append(lib, rot=72) == append(lib, rot=80) == append(lib, T=1 << 24) == ESHAPE
    assert append(lib, n_q=1025, qs=1 << 20) == append(lib, n_pos=1 << 31) == ESHAPE
    assert append(lib, qs=255) == append(lib, ks=127) == append(lib, vs=64) == append(lib, qs=1 << 31) == ESHAPE
    assert append(lib, qs=260) == append(lib, ks=132) == append(lib, dt=F32, qs=258) == EALIGN
    for name in ("q", "k", "v", "cos", "sin", "pos", "slots", "out"):
        assert append(lib, **{name: at(9) + 8}) == EALIGN
    assert append(lib, out=at(0)) == append(lib, out=at(1) + 128) == append(lib, out=at(20)) == EALIAS
    assert append(lib, c=cache(vc=at(20))) == append(lib, c=cache(ks=at(22) + 4096)) == append(lib, k=at(21)) == EALIAS
    assert append(lib, c=cache(kc=at(6))) == append(lib, c=cache(kc=at(3))) == EALIAS
    assert append(lib, T=0, q=None, out=None, k=None, v=None, slots=None, pos=None) == OK
    assert append(lib, T=0, c=cache(d=96)) == ESHAPE


def test_read_refusals(lib):
    assert read(lib, T=-1) == read(lib, dt=E4M3) == read(lib, slots=None) == read(lib, k=None, v=None) == EINVAL
    assert read(lib, T=1 << 24) == ESHAPE
    assert read(lib, k=at(0) + 8) == read(lib, v=at(1) + 4) == read(lib, slots=at(6) + 8) == EALIGN
    assert read(lib, v=at(0)) == read(lib, k=at(20)) == read(lib, v=at(6)) == EALIAS
    assert read(lib, T=0, slots=None, k=None, v=None) == OK


def test_attention_refusals(lib):
    assert attend(lib, T=-1) == attend(lib, B=0) == attend(lib, n_q=0) == attend(lib, max_q=-1) == EINVAL
    assert attend(lib, pages=0) == attend(lib, window=-1) == attend(lib, scale=0.0) == attend(lib, scale=-1.0) == EINVAL
    assert attend(lib, scale=float("nan")) == attend(lib, scale=float("inf")) == EINVAL
    for name in ("q", "lens", "table", "y"):
        assert attend(lib, **{name: None}) == EINVAL
        assert attend(lib, **{name: at(9) + 4}) == EALIGN
    assert attend(lib, cu=at(9) + 4) == attend(lib, lse=at(9) + 4) == attend(lib, qs=260) == EALIGN
    assert attend(lib, n_q=3) == attend(lib, n_q=1026, qs=1 << 20) == attend(lib, T=4) == attend(lib, qs=255) == ESHAPE
    assert attend(lib, T=1 << 24, B=1, cu=at(9)) == attend(lib, B=1 << 20, T=1 << 20) == ESHAPE
    assert attend(lib, T=1 << 22, n_q=512, qs=1 << 20, B=1, cu=at(9)) == attend(lib, pages=(1 << 25) + 1) == ESHAPE
    assert attend(lib, pages=1 << 25, T=1 << 19, B=1 << 19) == ESHAPE
    assert attend(lib, ws=None) == attend(lib, nb=0) == EWORKSPACE
    need = lib.kv4_attention_workspace_bytes(3, 3, 4, 2, 64, 1, 5, 32)
    assert attend(lib, nb=need - 1) == EWORKSPACE and attend(lib, ws=at(5) + 16) == EALIGN
    assert attend(lib, y=at(0)) == attend(lib, lse=at(3)) == attend(lib, y=at(22)) == attend(lib, ws=at(3)) == EALIAS
    assert attend(lib, y=at(2)) == attend(lib, lse=at(1)) == attend(lib, cu=at(3)) == attend(lib, ws=at(2)) == EALIAS
    assert attend(lib, T=0, B=3, cu=at(9), q=None, y=None, ws=None) == OK
    assert attend(lib, T=0, B=3) == ESHAPE  # a query a sequence


def test_workspace_sizes(lib):
    f = lib.kv4_attention_workspace_bytes
    assert f(0, 3, 4, 2, 64, 1, 5, 32) == f(3, 0, 4, 2, 64, 1, 5, 32) == f(3, 3, 4, 2, 96, 1, 5, 32) == 0
    assert f(3, 3, 3, 2, 64, 1, 5, 32) == f(3, 3, 4, 2, 64, 1, 5, 33) == f(3, 3, 4, 2, 64, 1, 0, 32) == 0
    for args in [(1, 1, 32, 8, 128, 1, 9, 32), (4000, 3, 32, 8, 128, 0, 400, 32), (64, 64, 16, 8, 256, 1, 400, 32)]:
        assert f(*args) > 0 and f(*args) % 256 == 0


def test_binding_refusals():
    """Made on the host: by kind, device and shape, each with its reason."""
    import qlora_linear_amd as q
    c = q.kv4_cache(3, 2, 64, device="cpu")
    assert [tuple(t.shape) for t in c] == [(3, 2, 32, 32), (3, 2, 1, 32, 2), (3, 2, 8, 128), (3, 2, 1, 32, 2)]
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(4, dtype=torch.int64)
    for f in (lambda: q.kv4_append(x, x, x, c, slots), lambda: q.kv4_read(c, slots),
              lambda: q.kv4_attention(x, c, slots[None].int(), slots.int())):
        with pytest.raises(ValueError, match="GPU"):
            f()
    for f in (lambda: q.kv4_read(None, slots), lambda: q.kv4_read(c[:3], slots), lambda: q.kv4_read((1, 2, 3, 4), slots)):
        with pytest.raises(ValueError, match="four tensors"):
            f()
    for bad in (dict(head_dim=96), dict(group=16), dict(group=128, head_dim=64), dict(page_size=16), dict(page_size=33),
                dict(n_pages=0), dict(n_kv=0)):
        with pytest.raises(ValueError):
            q.kv4_cache(**{**dict(n_pages=3, n_kv=2, head_dim=64, device="cpu"), **bad})


def test_scales_whose_power_of_two_form_overflows(lib):
    """The kernel multiplies by scale log2 e: infinite in float32 from 2.36e38 on, where every score would be no number."""
    for scale in (2.4e38, 3e38, 3.4e38):
        assert attend(lib, scale=scale) == EINVAL
    assert attend(lib, scale=2.3e38, ws=None) == EWORKSPACE and attend(lib, scale=1e-45, ws=None) == EWORKSPACE


def test_a_cache_that_no_call_takes_is_not_made():
    """The entry points' limits, when the cache is made and not at its first use."""
    import qlora_linear_amd as q
    make = lambda **kw: q.kv4_cache(**{**dict(n_pages=1, n_kv=1, head_dim=64, device="meta"), **kw})  # noqa: E731
    for bad in (dict(page_size=4128), dict(page_size=8192), dict(n_kv=1025), dict(n_pages=1 << 31), dict(n_pages=1 << 30, page_size=1024)):
        with pytest.raises(ValueError):
            make(**bad)
    assert make(page_size=4096)[0].shape == (1, 1, 4096, 32) and make(n_kv=1024)[0].shape[1] == 1024
