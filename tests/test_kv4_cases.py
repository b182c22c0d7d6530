"""What the GPU tests of the attention kernels run, shown on the host: that their batches reach every
kernel and every way of sharing the work, and that their reference finds a mistake."""
import numpy as np
import pytest

from oracle import kv4 as o
from tests import kv4_util as u
from tests.test_kv4_bounds import DIMS, most_nq

# ---- waves as workers --------------------------------------------------------------------
# One kernel to each (head_dim, group, 16-row tiles of a row block). Sequences' new tokens and keys are
# drawn up to `n` and `L`.
#   kind       cu_q and max_q: "one" a query each without cu_q, "bound", "free" (no bound: a launch lists the row blocks)
WAVES = []
for D, G in DIMS:
    WAVES += [(D, G, 1, "one", dict(B=70, n=1, heads=2, n_kv=16, L=150), 0), (D, G, 1, "free", dict(B=80, n=3, heads=4, n_kv=14, L=90), 20)]
    if most_nq(D, G) == 1:
        WAVES.append((D, G, 1, "bound", dict(B=24, n=20, heads=2, n_kv=16, L=120), 33))
    if most_nq(D, G) >= 2:
        WAVES += [(D, G, 2, "bound", dict(B=44, n=8, heads=3, n_kv=26, L=130), 40), (D, G, 2, "free", dict(B=50, n=10, heads=3, n_kv=24, L=100), 0)]
    if most_nq(D, G) == 2:
        WAVES.append((D, G, 2, "bound", dict(B=24, n=40, heads=2, n_kv=16, L=170), 0))
    if most_nq(D, G) == 4:
        WAVES += [(D, G, 4, "bound", dict(B=48, n=12, heads=5, n_kv=24, L=140), 0), (D, G, 4, "free", dict(B=20, n=70, heads=4, n_kv=13, L=200), 31),
                  (D, G, 4, "bound", dict(B=24, n=50, heads=2, n_kv=24, L=90), 25)]
# more row blocks and heads than workers, of few keys each: several to a worker
WAVES += [(128, 64, 2, "bound", dict(B=70, n=9, heads=2, n_kv=32, L=20), 0), (256, 128, 1, "one", dict(B=75, n=1, heads=1, n_kv=32, L=45), 0),
          (64, 32, 1, "one", dict(B=300, n=1, heads=3, n_kv=16, L=40), 0)]


def waves_batch(i):
    D, G, nq, kind, s, window = WAVES[i]
    g = np.random.default_rng(100 + i)
    seqs = []
    for b in range(s["B"]):
        n = 1 if kind == "one" else s["n"] if b % 8 else int(g.integers(0, s["n"] + 1))
        L = int(g.integers(0, s["L"] + 1)) if b % 5 else s["L"]
        seqs.append((n, L if b % 11 == 0 or kind == "one" else max(L, n)))
    batch = u.Batch(i, seqs, s["heads"] * s["n_kv"], s["n_kv"], D, G, (32, 64, 96)[i % 3])
    return batch, 1 if kind == "one" else s["n"] if kind == "bound" else 0, window


def test_every_kernel_of_waves_is_run():
    kernels, ways = set(), set()
    several = cut = 0
    for i, (D, G, nq, kind, *_) in enumerate(WAVES):
        batch, max_q, window = waves_batch(i)
        p = batch.plan(max_q)
        assert p["solo"] and p["nq"] == nq, WAVES[i]
        kernels.add((D, G, nq))
        ways.add((min(p["in_seq"], 2), p["by_head"], window > 0))
        shares = batch.shares(max_q, window)
        several += any(len(mine) > 2 for mine in shares)
        cut += any(not piece[-1] for mine in shares for piece in mine)
    assert kernels == {(D, G, nq) for D, G in DIMS for nq in (1, 2, 4) if nq <= most_nq(D, G)} and len(kernels) == 14
    # row blocks listed by a launch, by the workgroups (one and several a sequence); cuts by worker and by head
    assert {w[:2] for w in ways} == {(0, False), (1, False), (1, True), (2, False)}
    assert {w[0] for w in ways if w[2]} == {0, 1, 2}
    assert several >= 3 and cut >= len(WAVES) // 2


# ---- the reference -----------------------------------------------------------------------
@pytest.mark.parametrize("window", [0, 1, 9])
def test_reference_is_the_oracle(window):
    b = u.Batch(1, [(3, 40), (1, 0), (5, 2), (2, 70)], 6, 2, 64, 32, 32)
    for i, (n, L) in enumerate(b.seqs):
        y, lse, ey, el = b.reference(i, window=window)
        (kc, ks, kl), (vc, vs, vl) = b.parts(i)
        want, wl = o.attention(b.q[b.cu[i]:b.cu[i + 1]].astype(np.float64), o.values(kc, ks, kl, 32), o.values(vc, vs, vl, 32),
                               b.scale, window)
        want = np.moveaxis(want.reshape(n, 2, 3, 64), 1, 0).reshape(y.shape)
        wl = np.moveaxis(wl.reshape(n, 2, 3), 1, 0).reshape(lse.shape)
        np.testing.assert_allclose(y, want, rtol=1e-11, atol=1e-12)
        np.testing.assert_allclose(lse, wl, rtol=1e-12)
        assert np.all(ey <= 2.2 * u.UB * (np.abs(y) + 2.5)) and np.all(el <= 1e-3)
        one = b.reference(i, slice(1, 2), window)
        np.testing.assert_allclose(one[0], y[1:], rtol=1e-11, atol=1e-12)


def test_reference_without_some_keys():
    b = u.Batch(2, [(1, 96)], 2, 1, 64, 64, 32)
    y, lse, *_ = b.reference(0, missing=range(32, 64))
    (kc, ks, kl), (vc, vs, vl) = b.parts(0)
    keep = np.r_[0:32, 64:96]
    k, v = o.values(kc, ks, kl, 64)[keep], o.values(vc, vs, vl, 64)[keep]
    want, wl = o.attention(b.q.astype(np.float64), k, v, b.scale)
    np.testing.assert_allclose(y[0], want[0], rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(lse[0], wl[0], rtol=1e-12)


# ---- many tiles a wave ---------------------------------------------------------------------
# A wave's loop over tiles and pages at length, with scores that rise and fall by it. Key levels (powers of two of
# the weight) by sequence: spikes of 10, one in about 256 keys, over level keys, so that both weigh in the
# result; slow rises with a fall after each; slow falls with a rise. Values differ by level and place.
def spikes(b, t):
    return np.random.default_rng(1000 + b).integers(0, 257, 1 << 17)[t] == 0


def levels(b, t):
    if b % 3 == 0:
        return np.where(spikes(b, t), 10.0, 0.0)
    return (t if b % 3 == 1 else -t) % 2000 / 25.0


def centres(b, t):
    return np.where(spikes(b, t), -2.0, 2.0) if b % 3 == 0 else 2 * np.sin(t / 50)


LONG = [
    # sequences, query heads a key head, n_kv, D, group, page, window, max_q, waves as workers, what is checked of them
    ([(8, 20000 - 37 * b) for b in range(8)], 4, 4, 64, 32, 64, 0, 8, False, [(0, 1), (4, 3), (5, 0)]),
    ([(1, 26000 - 111 * b) for b in range(4)], 2, 8, 128, 64, 96, 0, 1, False, [(0, 2), (1, 7), (2, 0), (3, 5)]),
    ([(1, 9000 - 64 * b) for b in range(12)], 8, 8, 256, 128, 32, 7001, 1, False, [(0, 2), (1, 7), (2, 0), (3, 5)]),
    ([(200, 9000)] + [(1, 7000 - 100 * b) for b in range(8)], 4, 8, 128, 128, 256, 0, 0, False, [(0, 2), (1, 7), (2, 0), (3, 5), (0, 4)]),
    ([(1, 1900 + b) for b in range(64)], 3, 16, 64, 64, 32, 0, 1, True, [(0, 15), (1, 2), (2, 3), (63, 0), (33, 9)]),
    ([(5, 1500 - b) for b in range(66)], 5, 16, 64, 32, 64, 1333, 5, True, [(0, 15), (1, 2), (2, 3), (65, 0), (33, 9)]),
    ([(1, 700 + 5 * b) for b in range(65)], 1, 16, 256, 32, 128, 0, 1, True, [(0, 15), (1, 2), (2, 3), (63, 0), (33, 9)]),
]


def long_batch(i):
    seqs, heads, n_kv, D, G, page, window, max_q, solo, checked = LONG[i]
    batch = u.Batch(50 + i, seqs, heads * n_kv, n_kv, D, G, page, step=(0.04, 0.06), levels=levels, centres=centres)
    return batch, max_q, window, checked


def scores(batch, b, h, row, window):
    """Scores of a row of sequence b and key head h in powers of two, -inf where it does not see a key."""
    n, L = batch.seqs[b]
    (kc, ks, kl), _ = batch.parts(b, slice(h, h + 1))
    x = batch.scale / np.log(2) * (o.values(kc, ks, kl, batch.group)[:, 0] @ batch.rows(b, slice(h, h + 1))[0, row])
    last = L - n + row // (batch.n_q // batch.n_kv)
    t = np.arange(L)
    return np.where((t <= last) & (t > last - window if window else True), x, -np.inf)


@pytest.mark.parametrize("i", range(len(LONG)))
def test_long_loops_are_long(i):
    """At least eight tiles to nearly every wave, and maxima that are raised after its first tile."""
    batch, max_q, window, checked = long_batch(i)
    assert batch.plan(max_q)["solo"] == LONG[i][8]
    waves = list(batch.waves(max_q, window))
    steps = np.zeros((max(w[0] for w in waves) + 1, 4), int)
    for me, _, tiles in waves:
        steps[me, tiles[0] % 4 if not LONG[i][8] else 0] += len(tiles)
    per_wave = steps.reshape(-1) if not LONG[i][8] else steps[:, 0]
    assert np.median(per_wave) >= 8 and max(len(t) for *_, t in waves) >= 8
    raised = {}
    for b, h in checked:
        row0 = 0
        x = scores(batch, b, h, row0, window)
        raised[b, h] = sum(u.raises(x, tiles) for _, piece, tiles in waves if piece[:2] == (b, row0) and piece[3] == h)
    assert sum(raised.values()) >= 5 and any(raised[k] > 0 for k in raised if k[0] % 3 == 0)


def test_a_wrong_rescaling_is_found():
    """Sums that a raise leaves as they were, drops, or scales by the wrong power are off by more than the bound of
    the reference, on spikes and on a slow rise."""
    seqs = [(1, 12000)] * 2
    batch = u.Batch(9, seqs, 1, 1, 64, 64, 64, step=(0.04, 0.06), levels=levels, centres=centres)
    for b in range(2):
        x = scores(batch, b, 0, 0, 0)
        (_, (vc, vs, vl)) = batch.parts(b)
        v = o.values(vc, vs, vl, 64)[:, 0]
        waves = [range(s + w, min(s + 40, -(-len(x) // 32)), 4) for s in range(0, -(-len(x) // 32), 40) for w in range(4)]
        assert sum(u.raises(x, t) for t in waves) >= 10
        y, _, ey, _ = batch.reference(b)
        np.testing.assert_allclose(u.summed(x, v, waves), y[0, 0], rtol=1e-9, atol=1e-9)
        for wrong in (lambda rise: 1.0, lambda rise: 0.0, lambda rise: 2.0 ** rise, lambda rise: 2.0 ** (1 - rise)):
            assert np.any(np.abs(u.summed(x, v, waves, wrong) - y[0, 0]) > ey[0, 0]), b
