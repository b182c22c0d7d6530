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
