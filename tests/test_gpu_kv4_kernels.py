"""Every kernel of the paged 4-bit cache, against a float64 reference within a bound counted from
its roundings, in batches that are shown on the host to reach it."""
import numpy as np
import pytest
import torch

from oracle import kv4 as o
from tests import kv4_util as u
from tests import test_kv4_cases as cases

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import qlora_linear_amd as q
    q.library()
    return q


def attend(q, batch, max_q, window, **kw):
    """kv4_attention of a batch, with max_q as the C entry point takes it."""
    rows = {} if max_q == 1 and len(batch.seqs) == int(batch.cu[-1]) else dict(cu_q=torch.from_numpy(batch.cu).cuda(),
                                                                               max_q=max_q or None)
    return q.kv4_attention(*batch.device(), scale=batch.scale, window=window, return_lse=True, **rows, **kw)


@pytest.mark.parametrize("i", range(len(cases.WAVES)), ids=lambda i: "-".join(str(x) for x in cases.WAVES[i][:4]) + f"-{i}")
def test_waves_as_workers(q, i):
    batch, max_q, window = cases.waves_batch(i)
    print("waves", i, cases.WAVES[i], flush=True)
    y, lse = attend(q, batch, max_q, window)
    print("largest share of the bound", batch.check(y, lse, window), flush=True)
    again, _ = attend(q, batch, max_q, window)
    assert torch.equal(again, y)  # the result does not depend on the run


@pytest.mark.parametrize("i", range(len(cases.LONG)), ids=lambda i: f"{len(cases.LONG[i][0])}x{cases.LONG[i][0][0][1]}-" +
                         "-".join(str(x) for x in cases.LONG[i][1:8]))
def test_long_loops(q, i):
    """Many tiles and pages a wave; scores that rise and fall on the way."""
    batch, max_q, window, checked = cases.long_batch(i)
    print("long", i, cases.LONG[i][1:], flush=True)
    y, lse = attend(q, batch, max_q, window)
    for b, h in checked:
        print("share of the bound", b, h, batch.check(y, lse, window, [b], slice(h, h + 1)), flush=True)
    again, _ = attend(q, batch, max_q, window)
    assert torch.equal(again, y)


# ---- append: prompts -----------------------------------------------------------------------
# Tokens whose slots run on in scattered pages, as a prompt's do: values of four tokens at once.
# T, n_q, n_kv, D, group, page, rot, interleaved, dtype, first slot of the run
RUNS = [
    (600, 4, 3, 64, 32, 32, 64, False, torch.bfloat16, 0), (777, 2, 9, 64, 64, 96, 0, False, torch.float32, 4),
    (515, 3, 5, 128, 64, 64, 128, True, torch.bfloat16, 0), (1025, 4, 4, 128, 128, 32, 64, False, torch.float32, 28),
    (513, 2, 5, 256, 128, 32, 256, False, torch.bfloat16, 8), (801, 6, 2, 256, 32, 64, 16, True, torch.float32, 0),
    (640, 2, 2, 128, 32, 64, 128, False, torch.bfloat16, 1), (700, 1, 1, 64, 64, 32, 32, True, torch.bfloat16, 2),
    (999, 1, 2, 256, 64, 128, 0, False, torch.bfloat16, 31), (9001, 2, 2, 64, 32, 256, 64, False, torch.bfloat16, 8),
    (8192 + 514, 1, 1, 128, 64, 32, 0, False, torch.float32, 12),
]


@pytest.mark.parametrize("case", RUNS, ids=lambda c: "-".join(str(x).removeprefix("torch.") for x in c))
@pytest.mark.parametrize("broken", [False, True])
def test_append_runs(q, case, broken):
    """Stored codes and scales, bit for bit. broken: within fours of tokens some have no slot, the slot of
    another (of which the last is kept) or no position."""
    T, n_q, n_kv, D, group, page, rot, inter, dtype, first = case
    print("runs", case, broken, flush=True)
    g = np.random.default_rng(T + D + first)
    pages = (first + T - 1) // page + 4
    at = first + np.arange(T)
    slots = g.permutation(pages)[at // page] * page + at % page
    n_pos = T + 40
    pos = 37 + np.arange(T)
    if broken:
        for t in range(5, T, 37):  # (every place within four and within a tile)
            kind = t // 37 % 4
            if kind == 0:
                slots[t] = -1
            elif kind == 1:
                slots[t] = slots[t - 1 - t % 5]
            elif kind == 2:
                slots[t] = slots[min(t + 1, T - 1)]
            else:
                pos[t] = n_pos
    fours = sum(slots[t] % 4 == 0 and np.array_equal(slots[t:t + 4], slots[t] + np.arange(4)) for t in range(0, T - 3, 4))
    assert fours > T / 8 if first % 4 == 0 else fours == 0
    cache = q.kv4_cache(pages, n_kv, D, page, group)
    for t in cache:
        t.view(torch.uint8).random_(0, 250)
    before = tuple(t.float().cpu().numpy() if t.dtype is torch.bfloat16 else t.cpu().numpy() for t in cache)
    rows = [torch.from_numpy(g.standard_normal((T, n, D)).astype(np.float32)).to(dtype) for n in (n_q, n_kv, n_kv)]
    turned = [a.double().numpy() for a in rows]
    kw, placed = {}, np.ones(T, bool)
    if rot:
        angle = np.arange(n_pos)[:, None] * 1e4 ** (-np.arange(0, rot, 2) / rot)
        cos, sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
        kw = dict(cos=torch.from_numpy(cos).cuda(), sin=torch.from_numpy(sin).cuda(), positions=torch.from_numpy(pos).cuda(),
                  interleaved=inter)
        placed = pos < n_pos
        turned[:2] = [o.rotate(a, cos, sin, np.where(placed, pos, 0), inter) for a in turned[:2]]
    got = q.kv4_append(*(a.cuda() for a in rows), cache, torch.from_numpy(slots).cuda(), **kw)
    assert np.array_equal(got.float().cpu().numpy(), o.rounded(turned[0]) * placed[:, None, None])
    after = tuple(t.float().cpu().numpy() if t.dtype is torch.bfloat16 else t.cpu().numpy() for t in cache)
    last = {int(slots[t]): t for t in range(T) if placed[t] and slots[t] >= 0}
    keep, where = np.array(list(last.values())), np.array(list(last))
    for have, want in zip(o.read(after, where), (o.quantize(o.rounded(a[keep]), group) for a in turned[1:])):
        for a, b in zip(have, want):
            assert np.array_equal(a, b)
    others = np.setdiff1d(np.arange(pages * page), where)
    for have, want in zip(o.read(after, others), o.read(before, others)):
        for a, b in zip(have, want):
            assert np.array_equal(a, b, equal_nan=a.dtype.kind == "f")


# ---- attention: the one launch, values that are no numbers, missing pages ------------------
@pytest.mark.parametrize("D,G", cases.DIMS)
@pytest.mark.parametrize("n,heads", [(1, 4), (6, 4), (5, 13)])
@pytest.mark.parametrize("page,window", [(32, 0), (64, 100), (96, 0)])
def test_up_to_512_keys_in_one_launch(q, D, G, n, heads, page, window):
    width = 512 // page
    seqs = [(n, L) for L in (min(500, width * page), 0, 1, 33, width * page, 256)]
    batch = u.Batch(D + G + n, seqs, 2 * heads, 2, D, G, page, width=width)
    assert batch.plan(n)["whole"]
    print("one launch", D, G, n, heads, page, window, flush=True)
    y, lse = attend(q, batch, n, window)
    batch.check(y, lse, window)


@pytest.mark.parametrize("D,G,heads", [(64, 32, 2), (128, 128, 2), (256, 64, 3), (64, 64, 4)])
@pytest.mark.parametrize("key", [83, 20])  # one that some queries see, one in a tile that all see
def test_no_numbers_reach_every_query_that_sees_them(q, D, G, heads, key):
    """NaN or an infinity in a value's scales, NaN in a key's: no finite element in the rows of the queries that
    see it, the others' the same bits. (An infinite key may win or lose all of the weight.)"""
    batch = u.Batch(31, [(20, 90), (1, 40), (5, 5)], 2 * heads, 2, D, G, 32)
    x, cache, table, lens = batch.device()
    kw = dict(cu_q=torch.from_numpy(batch.cu).cuda())
    want = q.kv4_attention(x, cache, table, lens, **kw)
    batch.check(want)
    assert torch.isfinite(want.float()).all()
    first = max(0, key - 70)  # of sequence 0's queries, the first that sees it
    for which, bad in ((1, float("nan")), (3, float("nan")), (3, float("inf")), (3, float("-inf"))):
        for part in (slice(0, 2), slice(0, 1), slice(1, 2)):  # step and least value, one of them
            for h in range(2):
                changed = [t.clone() for t in cache]
                changed[which][int(table[0, key // 32]), h, :, key % 32, part] = bad
                y = q.kv4_attention(x, changed, table, lens, **kw)
                clean = torch.ones(26, 2 * heads, dtype=torch.bool)
                clean[first:20, h * heads:(h + 1) * heads] = False
                assert torch.equal(y[clean], want[clean]), (which, bad, part, h)
                assert not torch.isfinite(y[~clean].float()).any(), (which, bad, part, h)


@pytest.mark.parametrize("D,G,page", [(64, 64, 32), (128, 32, 64), (256, 128, 32)])
@pytest.mark.parametrize("window", [0, 90])
def test_a_missing_page_has_no_keys(q, D, G, page, window):
    batch = u.Batch(7, [(3, 5 * page + 9), (1, 2 * page)], 4, 2, D, G, page)
    x, cache, table, lens = batch.device()
    cu = torch.from_numpy(batch.cu).cuda()
    for pages, bad in (((1,), -1), ((0, 3), cache[0].shape[0]), ((5,), 2 ** 31 - 1), ((0, 1, 2, 3, 4), -2 ** 31)):
        broken = table.clone()
        broken[0, list(pages)] = bad
        print("missing", pages, bad, flush=True)
        y, lse = q.kv4_attention(x, cache, broken, lens, cu_q=cu, window=window, return_lse=True)
        batch.check(y, lse, window, [0], missing=[t for p in pages for t in range(p * page, min((p + 1) * page, 5 * page + 9))])
        batch.check(y, lse, window, [1])


@pytest.mark.parametrize("far", [2.0 ** 90, 2.0 ** -90])
def test_far_keys_and_values(q, far):
    """Keys and values of far magnitudes, whose scores are ordinary by the scale."""
    batch = u.Batch(3, [(1, 700), (4, 300)], 8, 2, 128, 64, 32, step=(0.2 * far, 0.4 * far), scale=0.1 / far)
    y, lse = attend(q, batch, 4, 0)
    batch.check(y, lse)


# ---- sizes at their ends -------------------------------------------------------------------
@pytest.mark.parametrize("seqs,n_q,n_kv,D,G,page", [
    ([(1, 9000), (3, 4097), (1, 1)], 4, 2, 64, 32, 4096), ([(1, 2500), (40, 1057)], 2, 2, 128, 64, 1056),
    ([(1, 70), (2, 33)], 1024, 1, 64, 64, 32), ([(1, 40), (1, 9)], 1024, 1024, 64, 32, 32), ([(3, 50)], 1024, 4, 256, 128, 32)])
@pytest.mark.parametrize("bounded", [True, False])
def test_largest_pages_and_heads(q, seqs, n_q, n_kv, D, G, page, bounded):
    batch = u.Batch(len(seqs) + n_q, seqs, n_q, n_kv, D, G, page)
    print("ends", seqs, n_q, n_kv, D, G, page, bounded, flush=True)
    y, lse = attend(q, batch, max(n for n, _ in seqs) if bounded else 0, 0)
    batch.check(y, lse)


def test_very_many_sequences(q):
    """Tokens of 100003 sequences, far more than a workgroup's threads, of one page each."""
    B, D = 100003, 64
    batch = u.Batch(1, [(1, 32)] * 40, 2, 1, D, 64, 32)
    _, cache, table, _ = batch.device()
    g = torch.Generator(device="cuda").manual_seed(2)
    which = torch.randint(0, 40, (B,), generator=g, device="cuda")
    lens = torch.randint(0, 33, (B,), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn(B, 2, D, generator=g, device="cuda").bfloat16()
    y, lse = q.kv4_attention(x, cache, table[which][:, :1].contiguous(), lens, return_lse=True)
    assert bool((y[lens == 0] == 0).all()) and bool((lse[lens == 0] == -float("inf")).all())
    at = [0, 1, 1023, 1024, 5000, 65535, 65536, B - 2, B - 1] + torch.randint(0, B, (300,), generator=g, device="cuda").tolist()
    # The same tokens by themselves: p s is rounded about another m, half a step of bf16 of s |c - 8| <= 3.2 each, and
    # y; a score is off by (2 64 + 8) U scale |q| |k|, |q| |k| at most 3 6 64 = 1152 with scale 1 / 8, each
    for i in at:
        one, l1 = q.kv4_attention(x[i:i + 1].clone(), cache, table[which[i:i + 1]][:, :1].contiguous(), lens[i:i + 1].clone(), return_lse=True)
        assert torch.allclose(one.float(), y[i:i + 1].float(), rtol=2 * u.UB, atol=2 * u.UB * 3.2) and \
            (int(lens[i]) == 0 or torch.allclose(l1, lse[i:i + 1], rtol=1e-6, atol=3e-3)), i


@pytest.mark.parametrize("bounded", [True, False])
def test_lists_of_no_rows(q, bounded):
    """Row lists that name no row leave every row as it was."""
    batch = u.Batch(5, [(3, 100), (2, 64)], 4, 2, 64, 32, 32)
    x, cache, table, lens = batch.device()
    for rows in ([0, 0, 0], [5, 5, 5], [2, 2, 2]):
        out = torch.full((5, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        cu = torch.tensor(rows, dtype=torch.int32, device="cuda")
        q.kv4_attention(x, cache, table, lens, cu_q=cu, max_q=3 if bounded else None, out=out)
        assert bool((out == 7).all()), rows


def test_more_rows_than_the_bound(q):
    """Rows past max_q may be left as they were; those before it are right, and nothing else is written."""
    batch = u.Batch(6, [(40, 300), (9, 64), (1, 20)], 6, 2, 128, 64, 32)
    x, cache, table, lens = batch.device()
    cu = torch.from_numpy(batch.cu).cuda()
    wide = torch.full((50 + 8, 6, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    q.kv4_attention(x, cache, table, lens, cu_q=cu, max_q=9, out=wide[4:54])
    assert bool((wide[:4] == 7).all()) and bool((wide[54:] == 7).all())
    want = q.kv4_attention(x, cache, table, lens, cu_q=cu, max_q=40)
    batch.check(want)
    got = wide[4:54].clone()
    got[9:40] = want[9:40]
    batch.check(got)


@pytest.mark.parametrize("T", [8192, 8193, 8200])
def test_append_at_the_end_of_a_launch(q, T):
    """A slot that a token of the last launch, of one token or of eight, has in common with earlier ones."""
    D, n_kv = 128, 2
    g = torch.Generator(device="cuda").manual_seed(T)
    k, v = (torch.randn(T, n_kv, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    slots = torch.arange(T, device="cuda")
    slots[T - 1], slots[8191], slots[8190] = 5, 5, 8191
    a, b = (q.kv4_cache(T // 32 + 1, n_kv, D, 32, 32) for _ in range(2))
    q.kv4_append(None, k, v, a, slots)
    last = {s: t for t, s in enumerate(slots.tolist())}
    keep = torch.tensor(sorted(last.values()), device="cuda")
    for part in keep.split(300):
        q.kv4_append(None, k[part], v[part], b, slots[part])
    assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("bound", [None, 12])
def test_captured_ragged(q, bound):
    """Ragged rows captured once and replayed as the rows' places and the lengths change in their tensors, with eager
    calls between, in a workspace that a decode of other sizes also uses."""
    plans = [[(12, 500), (0, 0), (3, 90), (1, 700)], [(1, 1), (12, 12), (2, 640), (1, 33)], [(0, 5), (0, 0), (0, 9), (16 - 4, 300)],
             [(5, 650), (5, 651), (5, 652), (1, 300)]]
    batches = [u.Batch(60 + i, s, 8, 2, 64, 32, 64, width=11) for i, s in enumerate(plans)]
    made = [b.device() for b in batches]
    T, pages = 16, max(m[1][0].shape[0] for m in made)
    cache = q.kv4_cache(pages, 2, 64, 64, 32)
    x, table = torch.zeros(T, 8, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 11, dtype=torch.int32, device="cuda")
    lens, cu = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda")
    need = q.kv4_attention_workspace_bytes(T, 4, 8, 2, 64, bound or 0, 11, 64)
    ws = torch.empty(max(need, q.kv4_attention_workspace_bytes(1, 1, 8, 2, 64, 1, 11, 64)), dtype=torch.uint8, device="cuda")

    def place(i):
        m, b = made[i], batches[i]
        x.zero_()
        x[:b.q.shape[0]] = m[0]
        for to, part in zip(cache, m[1]):
            to[:part.shape[0]] = part
        table.copy_(m[2].masked_fill(m[2] >= m[1][0].shape[0], -1))
        lens.copy_(m[3])
        cu.copy_(torch.from_numpy(b.cu))

    out = torch.zeros_like(x)
    run = lambda y, w: q.kv4_attention(x, cache, table, lens, cu_q=cu, max_q=bound, out=y, workspace=w)  # noqa: E731
    place(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(out, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out, ws)
    for n in range(9):
        i = (2 * n + n // 4) % 4
        place(i)
        rows = int(batches[i].cu[-1])
        want = run(torch.zeros_like(x), None)
        q.kv4_attention(x[:1].contiguous(), cache, table[:1].contiguous(), lens[:1].contiguous(), workspace=ws)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:rows], want[:rows]), (n, i)
        batches[i].check(out[:rows])
