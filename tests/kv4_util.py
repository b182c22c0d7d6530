"""Batches over a paged 4-bit cache, made on the host: inputs, attention in float64 with a bound
of its float32 and bf16 roundings, and the schedule by which the kernel shares the work out. No
GPU arithmetic; device copies are made on demand."""
import numpy as np

from oracle import kv4 as o
from oracle.norm_w4 import to_bf16
from tests.test_kv4_bounds import plan, step_at, units_of

U = 2.0 ** -24  # half a step of float32
UB = 2.0 ** -8  # half a step of bf16


class Batch:
    """Sequences (n new tokens, L keys) in scattered pages of a random cache. Slots that no sequence
    has hold NaN scales; past a sequence's end the table (`width` columns, or two more than the longest
    needs) names pages that do not exist. levels(b, t): what is added, in powers of two of the
    softmax's weight, to the scores of key t of sequence b, through the keys' least values (queries have
    mean 1 then); centres(b, t): to its values."""

    def __init__(self, seed, seqs, n_q, n_kv, D, group, page, width=None, step=(0.2, 0.4), levels=None, centres=None, scale=None):
        g = np.random.default_rng(seed)
        self.seqs, self.n_q, self.n_kv, self.D, self.group, self.page = seqs, n_q, n_kv, D, group, page
        self.scale = D ** -0.5 if scale is None else scale
        need = [-(-L // page) for _, L in seqs]
        pages = sum(need) + 3
        self.table = g.choice([-1, -(2 ** 31), pages, 2 ** 31 - 1], (len(seqs), max(need + [0]) + 2 if width is None else width))
        self.table = self.table.astype(np.int32)
        order = list(g.permutation(pages))
        scales = np.full((2, pages, n_kv, D // group, page, 2), np.nan, np.float32)
        for b, m in enumerate(need):
            self.table[b, :m] = [order.pop() for _ in range(m)]
            for i in range(m):
                n = min(page, seqs[b][1] - i * page)
                s = to_bf16(g.uniform(*step, (2, n_kv, D // group, n)).astype(np.float32))
                lo = s * (0.5 * g.standard_normal(s.shape) - 7.5)
                if levels is not None:
                    lo[0] += levels(b, i * page + np.arange(n)) * np.log(2) / (self.scale * D)
                if centres is not None:
                    lo[1] += centres(b, i * page + np.arange(n))
                scales[:, self.table[b, i], :, :, :n] = np.stack([s, to_bf16(lo.astype(np.float32))], -1)
        codes = lambda *s: np.frombuffer(g.bytes(int(np.prod(s)) * pages * n_kv), np.uint8).reshape(pages, n_kv, *s)  # noqa: E731
        self.np = codes(page, D // 2), scales[0], codes(page // 4, 2 * D), scales[1]
        self.cu = np.concatenate([[0], np.cumsum([n for n, _ in seqs])]).astype(np.int32)
        rows = g.standard_normal((self.cu[-1], n_q, D))
        self.q = to_bf16((rows * 2 if levels is None else 1 + 0.3 * rows).astype(np.float32))

    def device(self):
        """(q, cache, table, lens) as kv4_attention takes them."""
        import torch
        bf = lambda a: torch.from_numpy(a).cuda().bfloat16()  # noqa: E731
        at = lambda a: torch.from_numpy(np.array(a)).cuda()  # noqa: E731
        cache = at(self.np[0]), bf(self.np[1]), at(self.np[2]), bf(self.np[3])
        return bf(self.q), cache, at(self.table), at(np.array([L for _, L in self.seqs], np.int32))

    def parts(self, b, heads=slice(None)):
        """((codes, s, lo) of keys, of values) of sequence b and some key heads, [L, h, ..]."""
        kc, ks, vc, vs = self.np
        t = np.arange(self.seqs[b][1])
        slots = self.table[b, t // self.page].astype(np.int64) * self.page + t % self.page
        return o.read((kc[:, heads], ks[:, heads], vc[:, heads], vs[:, heads]), slots)

    def rows(self, b, heads=slice(None)):
        """Queries [h, n heads, D] of sequence b by key head, tokens slowest."""
        n = self.seqs[b][0]
        per = self.n_q // self.n_kv
        x = self.q[self.cu[b]:self.cu[b + 1]].astype(np.float64).reshape(n, self.n_kv, per, self.D)[:, heads]
        return np.moveaxis(x, 1, 0).reshape(x.shape[1], n * per, self.D)

    def reference(self, b, heads=slice(None), window=0, missing=()):
        """(y [h, n heads, D], lse, bounds of both) of sequence b; `missing` keys have no place."""
        n, L = self.seqs[b]
        G, groups = self.group, self.D // self.group
        qs = self.rows(b, heads)
        y, lse = np.zeros(qs.shape), np.full(qs.shape[:2], -np.inf)
        ey, el = np.zeros(y.shape), np.zeros(lse.shape)
        if qs.shape[1] == 0 or L == 0:
            return y, lse, ey, el
        rep = lambda a: np.repeat(a.astype(np.float64), G, -1)  # noqa: E731
        (kc, ks, kl), (vc, vs, vl) = self.parts(b, heads)
        by_head = lambda a: np.moveaxis(a, 1, 0)  # noqa: E731
        k, v = by_head(o.values(kc, ks, kl, G)), by_head(o.values(vc, vs, vl, G))
        k_size = by_head(kc * rep(ks) + np.abs(rep(kl)))
        dev = by_head(rep(vs) * np.abs(vc - 8.0))
        size = by_head(rep(vs) * (vc + 8.0) + np.abs(rep(vl) + 8 * rep(vs)))
        j = np.repeat(np.arange(n), self.n_q // self.n_kv)[:, None]
        t = np.arange(L)[None]
        seen = t <= L - n + j
        if window:
            seen &= t > L - n + j - window
        seen[:, list(missing)] = False
        some = seen.any(1)
        mT = lambda a: np.swapaxes(a, 1, 2)  # noqa: E731
        x = np.where(seen, self.scale * (qs @ mT(k)), -np.inf)
        top = np.where(some, x.max(-1), 0.0)
        p = np.exp(x - top[..., None])
        total = p.sum(-1)
        w = p / np.where(some, total, 1)[..., None]
        y = w @ v
        lse = np.where(some, top + np.log(np.where(some, total, 1)), -np.inf)
        # A score, in units of itself: the sums of a group's products (a matrix instruction may cut its
        # sums off, twice a rounding) and of its query's elements, three roundings of the scales, and 2 groups
        # fused additions whose partial sums hold m, at most the largest score (and the bar's 8 ln 2).
        # The difference from m and of two m (|x - top| and the bar), 2^x (4), one factor for each
        # raise, at most one a tile of 32 keys, and the joins'.
        d = np.where(seen, np.abs(x - top[..., None]), 0)
        most = np.abs(np.where(seen, x, 0)).max(-1) + 6
        rel = U * (self.scale * (2 * G + 2 * groups + 6) * (np.abs(qs) @ mT(k_size)) + (2 * groups + 2) * most[..., None] +
                   4 * (d + 12) + 4 * (L / 32 + 4) + 8)
        # sums over keys, of one key after another at the worst and twice a rounding, and of the parts
        adds = (2 * L + 128) * U
        el = (w * rel).sum(-1) + adds + 4 * U * (np.abs(np.where(some, lse, 0)) + most + 16)
        # y: the weights, l, p s to bf16 against c - 8, the sums of c and of 8 apart, y to bf16; weights, and
        # p s against |c - 8| <= 8, below the least normal float32
        ey = (w * rel) @ np.abs(v) + el[..., None] * np.abs(y) + UB * (w @ dev) + 2 * adds * (w @ size) + UB * np.abs(y)
        ey = ey + 2.0 ** -120 * size.sum(1)[:, None] + L * 2.0 ** -122
        return y, lse, np.where(some[:, None], 1.02 * ey, 0), np.where(some, 1.02 * el, 0)

    def check(self, y, lse=None, window=0, seqs=None, heads=slice(None), missing=()):
        """y and lse, as kv4_attention returned them, against the reference, of some sequences and key
        heads. Returns the largest share of its bound that an error of y takes."""
        have_y = y.float().cpu().numpy().reshape(self.q.shape[0], self.n_kv, self.n_q // self.n_kv, self.D)
        have_l = None if lse is None else lse.cpu().numpy().reshape(self.q.shape[0], self.n_kv, self.n_q // self.n_kv)
        worst = 0.0
        for b in range(len(self.seqs)) if seqs is None else seqs:
            want, wl, ey, el = self.reference(b, heads, window, missing)
            at = slice(self.cu[b], self.cu[b + 1])
            got = np.moveaxis(have_y[at][:, heads], 1, 0).reshape(want.shape)
            err = np.abs(got - want)
            assert np.all(err <= ey), (b, self.seqs[b], float((err / np.maximum(ey, 1e-30)).max()))
            worst = max(worst, float((err / np.maximum(ey, 1e-30)).max(initial=0)))
            if have_l is not None:
                got = np.moveaxis(have_l[at][:, heads], 1, 0).reshape(wl.shape)
                seen = np.isfinite(wl)
                assert np.array_equal(np.isfinite(got), seen) and np.all(got[~seen] == -np.inf), b
                assert np.all(np.abs(got[seen] - wl[seen]) <= el[seen]), b
        return worst

    # ---- the kernel's schedule ----
    def plan(self, max_q):
        """max_q as the C entry point takes it: 1 without cu_q, 0 without a bound."""
        return plan(int(self.cu[-1]), len(self.seqs), self.n_q, self.n_kv, self.D, max_q, self.table.shape[1] * self.page, self.group)

    def row_blocks(self, p, window=0):
        """(sequence, first row, rows, lo, hi) of every row block of the line, None for one that a
        sequence lacks."""
        heads, R, out = self.n_q // self.n_kv, 16 * p["nq"], []
        for b, (n, L) in enumerate(self.seqs):
            mine = -(-n * heads // R)
            for i in range(p["in_seq"] or mine):
                rows = min(R, n * heads - i * R)
                if i > 0 and rows <= 0:
                    out.append(None)
                    continue
                j0, j1 = i * R // heads, (i * R + max(rows, 1) - 1) // heads
                hi = max(L - n + j1 + 1, 0)
                lo = max(L - n + j0 + 1 - window, 0) if window else 0
                out.append((b, i * R, rows, *((lo, hi) if rows > 0 and lo < hi else (0, 0))))
        return out

    def shares(self, max_q, window=0):
        """Of each worker its pieces (sequence, first row, rows, key head, lo, hi, first step, last step, the
        whole row block)."""
        p = self.plan(max_q)
        blocks = self.row_blocks(p, window)
        if p["whole"]:
            return [[(*k[:3], h, *k[3:], 0, 1 << 20, True)] if k else [] for k in blocks for h in range(self.n_kv)]
        before = np.concatenate([[0], np.cumsum([units_of(*k[2:], p["cost"])[0] if k else 0 for k in blocks])])
        units = int(before[-1]) * self.n_kv
        workers = min(p["workers"], units)
        out = []
        for me in range(workers):
            at, end = me * units // workers, (me + 1) * units // workers
            item = int(np.searchsorted(before * self.n_kv, at, "right")) - 1
            mine = []
            while at < end:
                own = int(before[item + 1] - before[item])
                if own == 0:
                    item += 1
                    continue
                h, u0 = divmod(at - int(before[item]) * self.n_kv, own)
                u1 = min(own, u0 + end - at)
                b, row0, rows, lo, hi = blocks[item]
                mine.append((b, row0, rows, h, lo, hi, step_at(u0, rows, p["cost"]), step_at(u1, rows, p["cost"]),
                             u0 == 0 and u1 == own))
                at += u1 - u0
                if u1 == own and h == self.n_kv - 1:
                    item += 1
            out.append(mine)
        return out

    def waves(self, max_q, window=0):
        """Tiles that each wave works on of each piece: (worker, piece, the tiles)."""
        tiles = self.plan(max_q)["cost"][0]
        for me, mine in enumerate(self.shares(max_q, window)):
            for piece in mine:
                lo, hi, s0, s1 = piece[4:8]
                first, end = lo // 32 + tiles * s0, min(-(-hi // 32), lo // 32 + tiles * s1)
                for w in range(tiles):
                    if first + w < end:
                        yield me, piece, range(first + w, end, tiles)


def raises(x, tiles):
    """How often the maximum of a query that sees scores x (powers of two) is raised after the
    first keys that it sees, over a wave's tiles."""
    m, n = None, 0
    for t in tiles:
        top = x[32 * t:32 * t + 32].max(initial=-np.inf)
        if m is None:
            m = top if top > -np.inf else None
        elif top > m + 8:
            m, n = top, n + 1
    return n


def summed(x, v, waves, factor=lambda rise: 2.0 ** -rise):
    """The softmax of scores x (powers of two) over values v as the kernel forms it from the waves'
    tiles: a maximum a wave, raised past 8, sums that are rescaled by factor(rise), then joined."""
    parts = []
    for tiles in waves:
        m = l = None
        acc = np.zeros(v.shape[1])
        for t in tiles:
            s = x[32 * t:32 * t + 32]
            if m is None:
                m, l = s.max(), 0.0
            elif s.max() > m + 8:
                f = factor(s.max() - m)
                m, l, acc = s.max(), l * f, acc * f
            p = 2.0 ** (s - m)
            l, acc = l + p.sum(), acc + p @ v[32 * t:32 * t + 32]
        parts.append((m, l, acc))
    top = max(p[0] for p in parts)
    return sum(a * 2.0 ** (m - top) for m, _, a in parts) / sum(n * 2.0 ** (m - top) for m, n, _ in parts)
