"""The paged 4-bit cache on the GPU against the float64 oracle: rotated appends and rows read
back bit for bit, attention within a bound counted from its roundings."""
import math

import numpy as np
import pytest
import torch

from oracle import kv4 as o
from oracle.norm_w4 import to_bf16

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
U = 2.0 ** -24  # half a step of float32
UB = 2.0 ** -8  # half a step of bf16


@pytest.fixture(scope="module")
def q():
    import qlora_linear_amd as q
    q.library()
    return q


def host(t):
    return t.float().cpu().numpy()


def host_cache(c):
    return c[0].cpu().numpy(), host(c[1]), c[2].cpu().numpy(), host(c[3])


def tables(n_pos, rot, base=1e4):
    a = np.arange(n_pos)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


# ---- append and read ----------------------------------------------------------------
# T, n_q, n_kv, D, group, page, rot, interleaved, dtype
APPEND = [(1, 32, 8, 128, 128, 32, 128, False, BF), (5, 4, 4, 64, 32, 64, 32, True, F), (77, 6, 2, 256, 64, 96, 256, False, BF),
          (3, 1, 1, 64, 64, 32, 0, False, BF), (300, 12, 4, 128, 32, 32, 64, False, F), (530, 8, 8, 64, 64, 32, 64, True, BF),
          (2000, 3, 1, 128, 64, 256, 128, False, BF), (1025, 2, 2, 256, 128, 32, 16, False, F), (17, 7, 7, 256, 32, 4096, 48, True, BF)]


@pytest.mark.parametrize("T,n_q,n_kv,D,group,page,rot,inter,dtype", APPEND)
def test_append_and_read(q, T, n_q, n_kv, D, group, page, rot, inter, dtype):
    """Rotated queries, stored keys and values, bit for bit; slots that no token has keep what
    they hold; a token whose slot or position does not exist is left out."""
    print("append", T, n_q, n_kv, D, group, page, rot, inter, dtype, flush=True)
    g = np.random.default_rng(T + D)
    pages = 2 * T // page + 2
    cache = q.kv4_cache(pages, n_kv, D, page, group)
    for t in cache:
        t.view(torch.uint8).random_(0, 250)
    before = host_cache(cache)
    loud = 1 + 20 * (g.random((1, 1, D)) < 0.05)
    rows = [torch.from_numpy((g.standard_normal((T, n, D)) * loud).astype(np.float32)).to(dtype) for n in (n_q, n_kv, n_kv)]
    rows[1][0, 0, :group] = 0.5                                   # a group without range
    rows[2][T // 2] = torch.round(rows[2][T // 2])                # values on a grid: quotients at halves
    slots = g.permutation(pages * page)[:T]
    n_pos = 4096
    pos = g.integers(0, n_pos, T)
    if T > 2:
        slots[1], slots[T - 1] = -1, pages * page
        pos[2] = n_pos if T % 2 else -1
    kw, turned = {}, [host(a).astype(np.float64) for a in rows]
    placed = np.ones(T, bool)
    if rot:
        cos, sin = tables(n_pos, rot)
        kw = dict(cos=torch.from_numpy(cos).cuda(), sin=torch.from_numpy(sin).cuda(), positions=torch.from_numpy(pos).cuda(),
                  interleaved=inter)
        placed = (pos >= 0) & (pos < n_pos)
        turned[:2] = [o.rotate(a, cos, sin, np.where(placed, pos, 0), inter) for a in turned[:2]]
    got = q.kv4_append(*(a.cuda() for a in rows), cache, torch.from_numpy(slots).cuda(), **kw)
    want_q = o.rounded(turned[0]) * placed[:, None, None]
    assert got.dtype is BF and np.array_equal(host(got), want_q)

    ok = placed & (slots >= 0) & (slots < pages * page)
    parts = [o.quantize(o.rounded(a[ok]), group) for a in turned[1:]]
    after = host_cache(cache)
    for have, want in zip(o.read(after, slots[ok]), parts):
        for a, b in zip(have, want):
            assert np.array_equal(a, b)
    # every other slot as it was
    others = np.setdiff1d(np.arange(pages * page), slots[ok])
    for have, want in zip(o.read(after, others), o.read(before, others)):
        for a, b in zip(have, want):
            assert np.array_equal(a, b, equal_nan=a.dtype.kind == "f")
    # read back: one rounding of s c + lo to float32, one more to bf16
    at = torch.from_numpy(slots).cuda()
    for kind in (F, BF):
        for have, (c, s, lo) in zip(q.kv4_read(cache, at, kind), parts):
            v = o.values(c, s, lo, group).astype(np.float32)
            assert have.shape == (T, n_kv, D) and have.dtype is kind
            assert np.array_equal(host(have)[ok], v if kind is F else to_bf16(v))
            out = (slots < 0) | (slots >= pages * page)
            assert np.all(host(have)[out] == 0)


def test_append_wide_rows_and_no_queries(q):
    """Rows that are parts of a fused projection's output, and keys and values alone."""
    g = torch.Generator().manual_seed(1)
    T, n_q, n_kv, D = 40, 6, 2, 64
    wide = torch.randn(T, (n_q + 2 * n_kv) * D + 64, generator=g).bfloat16().cuda()
    parts = wide[:, :n_q * D], wide[:, n_q * D:(n_q + n_kv) * D], wide[:, (n_q + n_kv) * D:(n_q + 2 * n_kv) * D]
    cos, sin = (torch.from_numpy(t).cuda() for t in tables(64, D))
    kw = dict(cos=cos, sin=sin, positions=torch.arange(T + 3).cuda()[3:])  # starts at 8-byte offsets
    slots = torch.randperm(128, generator=g)[:T].cuda()
    one, two, three = (q.kv4_cache(4, n_kv, D, 32, 32) for _ in range(3))
    a = q.kv4_append(*parts, one, slots, **kw)
    b = q.kv4_append(*(p.contiguous().view(T, -1, D) for p in parts), two, slots, **kw)
    assert q.kv4_append(None, parts[1], parts[2], three, slots, **kw) is None
    assert a.shape == (T, n_q * D) and a.is_contiguous() and torch.equal(a.view(T, n_q, D), b)
    assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(one, two, three))


@pytest.mark.parametrize("T", [2, 40, 511, 512, 3000])
def test_append_keeps_the_last_of_a_slot(q, T):
    g = np.random.default_rng(T)
    D, n_kv = 64, 3
    k, v = (torch.from_numpy(g.standard_normal((T, n_kv, D)).astype(np.float32)).cuda() for _ in range(2))
    slots = g.integers(0, max(1, T // 3), T)
    pos = np.where(g.random(T) < 0.2, 99, 5)  # some tokens are left out and do not count
    pos[0] = 5
    cos, sin = (torch.from_numpy(t).cuda() for t in tables(9, D))
    a, b = (q.kv4_cache(T // 32 + 1, n_kv, D, 32, 64) for _ in range(2))
    q.kv4_append(None, k, v, a, torch.from_numpy(slots).cuda(), cos=cos, sin=sin, positions=torch.from_numpy(pos).cuda())
    last = {int(s): t for t, s in enumerate(slots) if pos[t] == 5}
    keep = torch.tensor(sorted(last.values()))
    q.kv4_append(None, k[keep], v[keep], b, torch.from_numpy(slots[keep.numpy()]).cuda(), cos=cos, sin=sin,
                 positions=torch.from_numpy(pos[keep.numpy()]).cuda())
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("far", [2.0 ** -130, 2.0 ** -120, 2.0 ** 120, 2.0 ** -60])
def test_append_far_values(q, far):
    """Ranges near the ends of bf16's: subnormal steps, reciprocals that overflow."""
    g = np.random.default_rng(9)
    x = to_bf16((g.standard_normal((8, 1, 64)) * far).astype(np.float32))
    x[3] = to_bf16(np.float32(far) * np.round(x[3] / np.float32(far)))
    x[4, 0, 1:] = 0
    t = torch.from_numpy(x).cuda()
    cache = q.kv4_cache(1, 1, 64, 32, 32)
    q.kv4_append(None, t, t, cache, torch.arange(8).cuda())
    want = o.quantize(x, 32)
    for part in o.read(host_cache(cache), np.arange(8)):
        for a, b in zip(part, want):
            assert np.array_equal(a, b)


# ---- attention ----------------------------------------------------------------------
class Batch:
    """Sequences (n new tokens, L keys) in pages of a random cache. Slots that no sequence has
    hold NaN scales, the table names pages that do not exist past each sequence's end."""

    def __init__(self, seed, seqs, n_q, n_kv, D, group, page, spread=2.0):
        g = self.g = np.random.default_rng(seed)
        self.seqs, self.group, self.D = seqs, group, D
        need = [-(-L // page) for _, L in seqs]
        pages = sum(need) + 3
        codes = lambda *s: g.integers(0, 256, (pages, n_kv, *s), dtype=np.uint8)  # noqa: E731
        scale = np.full((2, pages, n_kv, D // group, page, 2), np.nan, np.float32)
        order = list(g.permutation(pages))
        self.table = g.choice([-1, -(2 ** 31), pages, 2 ** 31 - 1], (len(seqs), max(need + [0]) + 2)).astype(np.int32)
        for b, m in enumerate(need):
            self.table[b, :m] = [order.pop() for _ in range(m)]
            for i in range(m):
                n = min(page, seqs[b][1] - i * page)
                s = to_bf16((0.2 + 0.2 * g.random((2, n_kv, D // group, n))).astype(np.float32))
                lo = to_bf16((s * (g.standard_normal(s.shape) - 7.5)).astype(np.float32))
                scale[:, self.table[b, i], :, :, :n] = np.stack([s, lo], -1)
        self.np = codes(page, D // 2), scale[0], codes(page // 4, 2 * D), scale[1]
        self.cache = tuple(torch.from_numpy(a).cuda().to(BF if a.dtype == np.float32 else torch.uint8) for a in self.np)
        self.cu = np.concatenate([[0], np.cumsum([n for n, _ in seqs])]).astype(np.int32)
        self.q = to_bf16((g.standard_normal((self.cu[-1], n_q, D)) * spread).astype(np.float32))
        self.args = [torch.from_numpy(self.q).cuda().bfloat16(), self.cache, torch.from_numpy(self.table).cuda(),
                     torch.tensor([L for _, L in seqs], dtype=torch.int32).cuda()]
        self.page = page

    def oracle(self, b, scale, window):
        """(y, lse, bounds of both) of sequence b. The bound counts: float32 roundings of a score
        (its D products and additions, and three), of 2^x and its argument, of the sums over keys
        (of a lane one after another, at most an eighth of the keys, and sixty to join), of p s to
        bf16 against c - 8, of y to bf16."""
        n, L = self.seqs[b]
        qs = self.q[self.cu[b]:self.cu[b + 1]].astype(np.float64)
        t = np.arange(L)
        (kc, ks, kl), (vc, vs, vl) = o.read(self.np, self.table[b, t // self.page] * self.page + t % self.page)
        k, v = o.values(kc, ks, kl, self.group), o.values(vc, vs, vl, self.group)
        y, lse = o.attention(qs, k, v, scale, window)
        rep = lambda a: np.repeat(a.astype(np.float64), self.group, -1)  # noqa: E731
        k_size = kc * rep(ks) + np.abs(rep(kl))
        dev = rep(vs) * np.abs(vc - 8.0)
        size = dev + np.abs(rep(vl) + 8 * rep(vs))
        ey, el = np.zeros(y.shape), np.zeros(lse.shape)
        heads = qs.shape[1] // k.shape[1]
        for j in range(n):
            hi = L - n + j + 1
            lo = max(0, hi - window) if window else 0
            if hi <= lo:
                continue
            for i in range(qs.shape[1]):
                h = i // heads
                x = scale * (k[lo:hi, h] @ qs[j, i])
                w = np.exp(x - lse[j, i])
                rel = scale * (self.D + 4) * U * (k_size[lo:hi, h] @ np.abs(qs[j, i]))
                rel = rel + 4 * U * (np.abs(x - x.max()) + 12) + 4 * U
                adds = (L / 8 + 64) * U
                el[j, i] = (w * rel).sum() + adds + 4 * U * np.abs(lse[j, i]) + 4 * U
                ey[j, i] = (w * rel) @ np.abs(v[lo:hi, h]) + el[j, i] * np.abs(y[j, i]) + UB * (w @ dev[lo:hi, h])
                ey[j, i] += 2 * adds * (w @ size[lo:hi, h]) + UB * np.abs(y[j, i]) + 2.0 ** -130
        return y, lse, 1.02 * ey, 1.02 * el

    def check(self, y, lse=None, scale=None, window=0, rows=None):
        y = host(y).reshape(self.q.shape)
        for b in range(len(self.seqs)):
            want, wl, ey, el = self.oracle(b, self.D ** -0.5 if scale is None else scale, window)
            at = slice(self.cu[b], self.cu[b + 1])
            err = np.abs(y[at] - want)
            assert np.all(err <= ey), (b, self.seqs[b], float((err / np.maximum(ey, 1e-30)).max()))
            if lse is not None:
                have, seen = host(lse)[at], np.isfinite(wl)
                assert np.array_equal(np.isfinite(have), seen) and np.all(have[~seen] == -np.inf)
                assert np.all(np.abs(have[seen] - wl[seen]) <= el[seen]), b


DECODE = [
    # lens, n_q, n_kv, D, group, page
    ([1], 4, 4, 64, 64, 32), ([1, 31, 32, 33], 8, 2, 128, 128, 32), ([500], 32, 8, 128, 128, 32),
    ([127, 0, 128, 129, 0], 8, 8, 64, 32, 64), ([700, 3, 255], 16, 1, 128, 64, 96), ([65, 300], 10, 2, 256, 128, 32),
    ([2500], 7, 7, 128, 32, 256), ([40] * 70, 4, 2, 64, 32, 32), ([1100, 9], 6, 2, 256, 32, 32), ([333], 24, 1, 64, 64, 32),
    ([90, 700], 40, 1, 128, 128, 64), ([200], 64, 1, 128, 64, 32), ([150, 20], 100, 1, 64, 32, 32), ([77] * 3, 12, 12, 256, 64, 32),
]


@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"{len(c[0])}x{max(c[0])}-{c[1]}-{c[2]}-{c[3]}-{c[4]}-{c[5]}")
@pytest.mark.parametrize("window", [0, 1, 50])
def test_decode(q, case, window):
    print("decode", case, window, flush=True)
    lens, *sizes = case
    b = Batch(len(lens) + max(lens), [(1, L) for L in lens], *sizes)
    y, lse = q.kv4_attention(*b.args, window=window, return_lse=True)
    b.check(y, lse, window=window)
    # the same through a list of rows, with and without its bound
    cu = torch.from_numpy(b.cu).cuda()
    for most in (1, None):
        y2, lse2 = q.kv4_attention(*b.args, cu_q=cu, max_q=most, window=window, return_lse=True)
        b.check(y2, lse2, window=window)
    again = q.kv4_attention(*b.args, window=window)
    assert torch.equal(again, y)  # the result does not depend on the run


RAGGED = [
    # (new tokens, keys), n_q, n_kv, D, group, page
    ([(5, 300), (5, 5), (5, 1000)], 16, 2, 128, 64, 32), ([(1, 100), (40, 600), (0, 50), (3, 33)], 8, 2, 128, 128, 64),
    ([(150, 150), (64, 200)], 4, 4, 64, 32, 32), ([(7, 3), (9, 0), (2, 2)], 6, 3, 64, 64, 32), ([(33, 70)], 5, 1, 256, 64, 96),
    ([(200, 333)], 12, 4, 256, 128, 32), ([(0, 7), (0, 0), (1, 1)], 4, 2, 128, 32, 32), ([(100, 1500)], 20, 4, 128, 32, 128),
    ([(70, 90), (1, 2000)], 3, 1, 256, 32, 32),
]


@pytest.mark.parametrize("case", RAGGED, ids=lambda c: "-".join(f"{n}of{L}" for n, L in c[0]) + f"-{c[1]}-{c[2]}-{c[3]}-{c[4]}")
@pytest.mark.parametrize("window", [0, 1, 37])
@pytest.mark.parametrize("bounded", [True, False])
def test_ragged(q, case, window, bounded):
    print("ragged", case, window, bounded, flush=True)
    seqs, *sizes = case
    b = Batch(sum(n + L for n, L in seqs), seqs, *sizes)
    y, lse = q.kv4_attention(*b.args, cu_q=torch.from_numpy(b.cu).cuda(), max_q=max(n for n, _ in seqs) if bounded else None,
                             window=window, return_lse=True)
    b.check(y, lse, window=window)


def test_many_sequences(q):
    """More sequences than a workgroup sums the steps of itself."""
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 200, 1500)]
    b = Batch(7, [(1, L) for L in lens], 2, 1, 64, 64, 32)
    y, lse = q.kv4_attention(*b.args, return_lse=True)
    b.check(y, lse)


def test_scale_and_large_scores(q):
    """Scores of hundreds, one key that takes all of the weight, falling and rising maxima."""
    for scale, spread in ((0.01, 1.0), (1.0, 6.0), (8.0, 1.0)):
        b = Batch(int(100 * scale), [(1, 800), (1, 65)], 4, 2, 128, 64, 32, spread)
        y, lse = q.kv4_attention(*b.args, scale=scale, return_lse=True)
        b.check(y, lse, scale=scale)


def test_no_numbers_stay_where_they_are(q):
    """A query of NaN or infinities gives no numbers in its own rows only; a key or value of such,
    in those of the queries that see it only."""
    seqs = [(20, 90), (1, 40), (5, 5)]
    b = Batch(31, seqs, 4, 2, 64, 32, 32)
    cu = torch.from_numpy(b.cu).cuda()
    want = q.kv4_attention(*b.args, cu_q=cu)
    x = b.args[0].clone()
    x[3, 1], x[22, 2] = float("nan"), float("inf")
    y = q.kv4_attention(x, *b.args[1:], cu_q=cu)
    same = torch.ones(26, 4, dtype=torch.bool)
    same[3, 1] = same[22, 2] = False
    assert torch.equal(y[same], want[same]) and not torch.isfinite(y[~same].float()).any()
    for which, bad in ((1, float("nan")), (3, float("nan")), (1, float("inf")), (3, float("-inf"))):
        for head in range(2):
            cache = [t.clone() for t in b.cache]
            at = 83  # sequence 0's queries from its 13th on see this key
            cache[which][int(b.table[0, at // 32]), head, :, at % 32] = bad
            y = q.kv4_attention(b.args[0], cache, *b.args[2:], cu_q=cu)
            clean = torch.ones(26, 4, dtype=torch.bool)
            clean[13:20, 2 * head:2 * head + 2] = False
            assert torch.equal(y[clean], want[clean]), (which, bad, head)
            assert which == 1 or not torch.isfinite(y[~clean].float()).any()


def test_rows_left_alone_and_strides(q):
    """Queries as part of a wider matrix; rows of no sequence, before and behind, are not written."""
    b = Batch(11, [(3, 200), (1, 90)], 8, 2, 64, 32, 32)
    cu = torch.from_numpy(b.cu + 2).cuda()
    T = int(b.cu[-1]) + 7
    wide = torch.full((T, 8 * 64 + 96), 9.0, dtype=BF).cuda()
    part = wide[:, 32:32 + 8 * 64]
    part[2:2 + int(b.cu[-1])] = b.args[0].flatten(1)
    out = torch.full((T, 8 * 64), 7.0, dtype=BF).cuda()
    y = q.kv4_attention(part, *b.args[1:], cu_q=cu, out=out)
    assert y is out
    b.check(y[2:2 + int(b.cu[-1])])
    assert bool((out[:2] == 7).all()) and bool((out[2 + int(b.cu[-1]):] == 7).all())


def test_pages_out_of_range_and_bad_lists(q):
    """A page that does not exist has no keys; lengths and row lists beyond their operands are cut
    to them, with guard bands around the outputs."""
    from tests.gpu_util import Guarded
    b = Batch(13, [(1, 96), (1, 64)], 4, 2, 64, 64, 32)
    y0 = q.kv4_attention(*b.args)
    table = b.args[2].clone()
    table[0, 1] = b.cache[0].shape[0]
    shorter = Batch(13, [(1, 96), (1, 64)], 4, 2, 64, 64, 32)
    y = q.kv4_attention(b.args[0], b.cache, table, b.args[3])
    # the same as with that page's keys gone: its neighbours close up
    closed = b.args[2].clone()
    closed[0, 1] = closed[0, 2]
    want = q.kv4_attention(b.args[0], b.cache, closed, torch.tensor([64, 64], dtype=torch.int32).cuda())
    assert torch.allclose(y.float(), want.float(), atol=2e-2) and torch.equal(y[1], y0[1])
    del shorter
    lens = torch.tensor([2 ** 31 - 1, -5], dtype=torch.int32).cuda()
    full = q.kv4_attention(b.args[0], b.cache, b.args[2], lens)
    assert torch.isfinite(full.float()[0]).all() and bool((full[1] == 0).all())
    lib = q.library()
    from tests.test_kv4_abi import Cache
    import ctypes
    c = Cache(b.cache[0].shape[0], 32, 2, 64, 64, *(t.data_ptr() for t in b.cache))
    need = lib.kv4_attention_workspace_bytes(2, 2, 4, 2, 64, 0, b.table.shape[1], 32)
    for rows in ([0, 1, 2], [5, 9, 2 ** 31 - 1], [-7, 2 ** 31 - 1, 0], [2, 1, 0], [0, 2, 2], [-2 ** 31, 2, 1]):
        print("rows", rows, flush=True)
        y, ws, lse = Guarded(2 * 4 * 64 * 2), Guarded(need), Guarded(2 * 4 * 4)
        cu = torch.tensor(rows, dtype=torch.int64).to(torch.int32).cuda()
        st = lib.kv4_attention(2, 2, 4, b.args[0].data_ptr(), 256, cu.data_ptr(), 0, b.args[3].data_ptr(), b.args[2].data_ptr(),
                               b.table.shape[1], 0, 0.125, ctypes.byref(c), y.ptr, lse.ptr, ws.ptr, need,
                               torch.cuda.current_stream().cuda_stream)
        assert st == 0
        torch.cuda.synchronize()
        assert y.canaries_intact() and ws.canaries_intact() and lse.canaries_intact()


def test_far_pages(q):
    """Byte offsets past 2^32 in codes and scales."""
    pages, n_kv, D, page = 70000, 8, 128, 128
    cache = q.kv4_cache(pages, n_kv, D, page, 128)
    assert cache[0].numel() > 2 ** 32
    g = torch.Generator().manual_seed(2)
    T = 300
    k, v = (torch.randn(T, n_kv, D, generator=g).bfloat16().cuda() for _ in range(2))
    far = torch.tensor([pages - 1, 3, pages - 2], dtype=torch.int32).cuda()
    t = torch.arange(T).cuda()
    slots = far[t // page].long() * page + t % page
    q.kv4_append(None, k, v, cache, slots)
    near = q.kv4_cache(4, n_kv, D, page, 128)
    q.kv4_append(None, k, v, near, t)
    for a, b in zip(q.kv4_read(cache, slots), q.kv4_read(near, t)):
        assert torch.equal(a, b)
    x = torch.randn(1, 32, D, generator=g).bfloat16().cuda()
    L = torch.tensor([T], dtype=torch.int32).cuda()
    a = q.kv4_attention(x, cache, far[None], L)
    b = q.kv4_attention(x, near, torch.arange(3, dtype=torch.int32)[None].cuda(), L)
    assert torch.equal(a, b)


# ---- together -----------------------------------------------------------------------
def layer(q, seed=0, d=256, n_q=4, n_kv=2, D=64):
    g = torch.Generator().manual_seed(seed)
    w = [torch.randn(n, k, generator=g).mul_(k ** -0.5).cuda() for n, k in ((n_q * D, d), (n_kv * D, d), (n_kv * D, d), (d, n_q * D))]
    packed = [q.w4_quantize(a, 64) for a in w]
    norm = (1 + 0.1 * torch.randn(d, generator=g)).bfloat16().cuda()
    cos, sin = (torch.from_numpy(t).cuda() for t in tables(512, D))

    def step(x, cache, slots, positions, table, lens, **kw):
        rows, scale, _ = q.rmsnorm_fwd_quant(x, norm)
        qkv = q.w4_matvec_multi(rows, *([p[i] for p in packed[:3]] for i in range(2)), x_scale=scale)
        turned = q.kv4_append(*qkv, cache, slots, cos=cos, sin=sin, positions=positions)
        y = q.kv4_attention(turned, cache, table, lens, **kw)
        return q.w4_matvec(y, *packed[3]), y, turned, qkv

    return step


def test_prompt_then_tokens(q):
    """A layer as it is served: a prompt of two sequences at once, then token by token, against the
    oracle's attention over the cache as it stands."""
    n_q, n_kv, D, d, page = 4, 2, 64, 256, 32
    step = layer(q)
    g = torch.Generator().manual_seed(5)
    cache = q.kv4_cache(9, n_kv, D, page, 64)
    table = torch.tensor([[7, 2, 0, 5], [1, 8, 3, 4]], dtype=torch.int32)
    lens = [70, 37]

    def slots_of(b, t):
        return table[b].long()[t // page] * page + t % page

    def against(y, turned, cu, lens):
        (kc, ks, kl), (vc, vs, vl) = o.read(host_cache(cache), np.arange(9 * page))
        k, v = o.values(kc, ks, kl, 64), o.values(vc, vs, vl, 64)
        for b in range(2):
            at = slots_of(b, torch.arange(lens[b])).numpy()
            want, _ = o.attention(host(turned).reshape(-1, n_q, D)[cu[b]:cu[b + 1]].astype(np.float64), k[at], v[at], D ** -0.5)
            have = host(y).reshape(-1, n_q, D)[cu[b]:cu[b + 1]]
            # p s (c - 8) rounded to bf16 and y to bf16, of values up to the largest
            assert np.abs(have - want).max() <= 2 * UB * max(np.abs(want).max(), np.abs(v[at]).max())

    x = torch.randn(sum(lens), d, generator=g).bfloat16().cuda()
    at = [torch.arange(n) for n in lens]
    cu = [0, 70, 107]
    out, y, turned, qkv = step(x, cache, torch.cat([slots_of(b, at[b]) for b in range(2)]).cuda(), torch.cat(at).cuda(),
                               table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                               cu_q=torch.tensor(cu, dtype=torch.int32).cuda())
    against(y, turned, cu, lens)
    assert out.shape == (107, d) and torch.isfinite(out.float()).all()
    for _ in range(3):
        lens = [n + 1 for n in lens]
        pos = torch.tensor([n - 1 for n in lens])
        x = torch.randn(2, d, generator=g).bfloat16().cuda()
        out, y, turned, qkv = step(x, cache, torch.stack([slots_of(b, pos[b]) for b in range(2)]).cuda(), pos.cuda(), table.cuda(),
                                   torch.tensor(lens, dtype=torch.int32).cuda())
        against(y, turned, [0, 1, 2], lens)


def test_captured_step(q):
    """A decode step captured once and replayed as positions, lengths and slots move on in their
    tensors, with the program's own calls between, against the same step made eagerly; two
    graphs that share a workspace."""
    step = layer(q)
    B, d, page = 3, 256, 32
    g = torch.Generator().manual_seed(6)
    start = [40, 3, 64]
    table = torch.tensor([[0, 5, 6], [1, 7, 8], [2, 3, 4]], dtype=torch.int32).cuda()
    one, two = (q.kv4_cache(9, 2, 64, page, 32) for _ in range(2))
    for c in (one, two):
        gen = torch.Generator().manual_seed(1)
        k = torch.randn(9 * page, 2, 64, generator=gen).bfloat16().cuda()
        q.kv4_append(None, k, k * 0.5, c, torch.arange(9 * page).cuda())
    ws = torch.empty(q.kv4_attention_workspace_bytes(B, B, 4, 2, 64, 1, 3, page), dtype=torch.uint8, device="cuda")
    x = torch.randn(B, d, generator=g).bfloat16().cuda()
    lens = torch.tensor(start, dtype=torch.int32).cuda()
    pos, slots = lens.long() - 1, torch.zeros(B, dtype=torch.int64).cuda()

    def run(cache, workspace=None):
        return step(x, cache, slots, pos, table, lens, workspace=workspace)[:2]

    def place(n):
        at = torch.tensor(start) + n
        lens.copy_(at.int())
        pos.copy_(at - 1)
        slots.copy_(table.cpu().long()[torch.arange(B), (at - 1) // page] * page + (at - 1) % page)

    place(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(one, ws)
    run(two)  # (the token of the call before the capture, in both caches)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(run(one, ws))
        graphs.append(graph)
    for n in range(1, 6):
        place(n)
        x.copy_(torch.randn(B, d, generator=g).bfloat16())
        want = run(two)
        (x.float().sum() + 1).item()
        graphs[n % 2].replay()
        graphs[1 - n % 2].replay()
        torch.cuda.synchronize()
        for have in outs:
            for a, b in zip(have, want):
                assert torch.equal(a, b), n
        assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_streams(q):
    """Two batches on two streams at once, each in its own workspace, against the same one after
    the other."""
    bs = [Batch(21, [(1, 900), (1, 1400)], 8, 2, 128, 64, 32), Batch(22, [(4, 800), (9, 1000)], 8, 2, 128, 64, 32)]
    kw = [{}, dict(cu_q=torch.from_numpy(bs[1].cu).cuda())]
    want = [q.kv4_attention(*b.args, **k) for b, k in zip(bs, kw)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    have = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                have[i].append(q.kv4_attention(*bs[i].args, **kw[i]))
    torch.cuda.synchronize()
    for h, w in zip(have, want):
        assert all(torch.equal(a, w) for a in h)


def test_refusals_on_gpu(q):
    c = q.kv4_cache(3, 2, 64)
    x = torch.zeros(4, 2, 64, dtype=BF).cuda()
    s = torch.arange(4).cuda()
    t, n = torch.zeros(4, 3, dtype=torch.int32).cuda(), torch.ones(4, dtype=torch.int32).cuda()
    cos = torch.zeros(5, 32).cuda()
    for f in (lambda: q.kv4_append(x, x, x[:3], c, s), lambda: q.kv4_append(x, x, x, c, s.int()),
              lambda: q.kv4_append(x, x.float(), x, c, s), lambda: q.kv4_append(x, x[:, :1], x, c, s),
              lambda: q.kv4_append(x, x, x, c, s[:3]), lambda: q.kv4_append(x, x, x, c, s, cos=cos),
              lambda: q.kv4_append(x, x, x, c, s, cos=cos[:, :20], sin=cos[:, :20], positions=s),
              lambda: q.kv4_append(x, x, x, c, s, cos=cos, sin=cos[:4], positions=s),
              lambda: q.kv4_append(x.transpose(0, 1), x, x, c, s), lambda: q.kv4_append(x.half(), x.half(), x.half(), c, s),
              lambda: q.kv4_read(c, s, torch.float16), lambda: q.kv4_read(c, s.view(2, 2)),
              lambda: q.kv4_attention(x.float(), c, t, n), lambda: q.kv4_attention(x, c, t.long(), n),
              lambda: q.kv4_attention(x, c, t, n[:3]), lambda: q.kv4_attention(x, c, t[:2], n[:2]),
              lambda: q.kv4_attention(x, c, t, n, cu_q=n), lambda: q.kv4_attention(x, c, t[:, :0], n),
              lambda: q.kv4_attention(x, c, t[:1], n[:1], cu_q=n[:2], max_q=0),
              lambda: q.kv4_attention(x, c, t, n, workspace=torch.zeros(1 << 20)),
              lambda: q.kv4_read((c[0], c[1], c[3], c[2]), s), lambda: q.kv4_read((*c[:3], c[3].cpu()), s)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: q.kv4_attention(x, c, t, n, scale=0.0), lambda: q.kv4_attention(x, c, t, n, window=-1),
              lambda: q.kv4_attention(x[:, :1].contiguous(), c, t, n),
              lambda: q.kv4_attention(x, c, t, n, out=x), lambda: q.kv4_attention(x, c, t, n, workspace=torch.zeros(256, dtype=torch.uint8).cuda())):
        with pytest.raises(q.LoraNF4Error):
            f()
    empty = x[:0]
    assert q.kv4_append(empty, empty, empty, c, s[:0]).shape == (0, 2, 64)
    assert q.kv4_read(c, s[:0])[0].shape == (0, 2, 64)
    assert q.kv4_attention(empty, c, t, n, cu_q=torch.zeros(5, dtype=torch.int32).cuda()).shape == (0, 2, 64)


def test_large_windows_are_refused(q):
    c = q.kv4_cache(3, 2, 64)
    x = torch.zeros(4, 2, 64, dtype=BF).cuda()
    t, n, cu = torch.zeros(4, 3, dtype=torch.int32).cuda(), torch.ones(4, dtype=torch.int32).cuda(), torch.arange(5, dtype=torch.int32).cuda()
    for kw in (dict(window=2 ** 31), dict(window=2 ** 32), dict(window=2 ** 32 + 5), dict(window=-2 ** 32 + 5),
               dict(cu_q=cu, max_q=2 ** 32 + 1)):
        with pytest.raises(ValueError, match="2\\^31"):
            q.kv4_attention(x, c, t, n, **kw)
    q.kv4_attention(x, c, t, n, window=2 ** 31 - 1)


@pytest.mark.parametrize("dtype", [BF, F])
def test_append_many_tokens_of_few_slots(q, dtype):
    """Tokens that go in several launches: the last of a slot, wherever it is, and every query."""
    T, D, n_q, n_kv, n = 70001, 64, 3, 2, 2000
    g = torch.Generator(device="cuda").manual_seed(5)
    x, k, v = (torch.randn(T, h, D, generator=g, device="cuda").to(dtype) for h in (n_q, n_kv, n_kv))
    slots = torch.randint(-1, n, (T,), generator=g, device="cuda")
    slots[-1] = slots[7]
    pos = torch.randint(0, 11, (T,), generator=g, device="cuda")  # (9 and 10 are in no table)
    cos, sin = (torch.from_numpy(t).cuda() for t in tables(9, D))
    a, b = (q.kv4_cache(n // 32 + 1, n_kv, D) for _ in range(2))
    y = q.kv4_append(x, k, v, a, slots, cos=cos, sin=sin, positions=pos)
    last = {s: t for t, (s, p) in enumerate(zip(slots.tolist(), pos.tolist())) if s >= 0 and p < 9}
    keep = torch.tensor(sorted(last.values())).cuda()
    q.kv4_append(None, k[keep], v[keep], b, slots[keep], cos=cos, sin=sin, positions=pos[keep])
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    for i in range(0, T, 500):  # (calls of one launch)
        e = slice(i, min(i + 500, T))
        assert torch.equal(y[e], q.kv4_append(x[e], k[e], v[e], b, slots[e], cos=cos, sin=sin, positions=pos[e]))
