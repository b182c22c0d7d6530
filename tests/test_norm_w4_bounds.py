"""Host-side model of the addressing of the norm and the packed-weight kernels (CPU).

As test_load_bounds.py does for the tiled kernels: the functions restate the index arithmetic
of rms_norm.hip, w4_quant.hip and w4_matvec.hip and check that every access lies inside its
operand, workspace or LDS array, that every output element is written exactly once and that a
buffer load needs no range check. They mirror the device code; a change to one changes its
model here. Workspace sizes come from the library itself."""
import os

import numpy as np
import pytest

from tests.test_load_bounds import Checker, boundary

ELEMS = {"bf16": 8, "f32": 4}  # of a 16-byte vector


@pytest.fixture(scope="module")
def lib():
    import qlora_linear_amd as q
    if not os.path.exists(q.library_path):
        from qlora_linear_amd import build
        build.build()
    return q.library()


# ---- norm (rms_norm.hip) ------------------------------------------------------------
def row_shape(T, vecs, most):
    if vecs <= 64:
        return 64, 1
    if vecs <= 128 and T > 512:
        return 64, 2
    if vecs <= 256:
        return 256, 1
    if vecs <= 512:
        return 256, 2
    nv = 1
    while nv <= most:
        if vecs <= 1024 * nv:
            return 1024, nv
        nv *= 2
    return 0, 0


def row_vectors(tpr, nv, d, kn):
    """Lengths of the vectors that the threads of a row load: all of the row, each once."""
    at = (np.arange(tpr)[:, None] + tpr * np.arange(nv)[None]).ravel() * kn
    left = np.clip(d - at, 0, kn)
    hit = np.zeros(d, np.int64)
    for j in range(kn):
        np.add.at(hit, at[left > j] + j, 1)
    assert (hit == 1).all()


WIDTHS = [1, 7, 64, 511, 512, 513, 1001, 1024, 1025, 2047, 2049, 4096, 4097, 8191, 8193, 16384, 16385, 32767, 32768]


@pytest.mark.parametrize("kind", ELEMS)
@pytest.mark.parametrize("quant", [False, True])
def test_norm_forward_rows(kind, quant):
    kn = ELEMS[kind]
    most = (16 if kn == 8 and quant else 32) // kn
    for d in WIDTHS:
        for T in (1, 512, 513, 1030):
            tpr, nv = row_shape(T, -(-d // kn), most)
            if tpr == 0:
                assert d > 1024 * kn * most
                continue
            row_vectors(tpr, nv, d, kn)
            rows = 256 // tpr if tpr < 256 else 1
            assert tpr * rows <= 1024 and rows * -(-T // rows) >= T
            assert tpr == 64 or rows == 1  # a barrier runs in workgroups of one row only


@pytest.mark.parametrize("kind", ELEMS)
def test_norm_backward_rows_and_workspace(lib, kind):
    kn = ELEMS[kind]
    for d in WIDTHS + [20000, 40001]:
        for T in (1, 3, 511, 512, 513, 1024, 1537, 4097, 9000):
            vecs = -(-d // kn)
            tpr, nv = row_shape(T, vecs, 16 // kn)
            part_rows = lib.rmsnorm_bwd_workspace_bytes(T, d) // (4 * d)  # rows of partial sums that fit
            limit = min(T, 512)
            assert part_rows >= limit
            if tpr == 0:  # dw in a pass of its own: rows b, b + blocks, ... of block b
                blocks = min(limit, 64)
                at = np.arange(-(-vecs // 256) * 256) * kn
                assert (np.clip(d - at, 0, kn).sum() == d) and blocks <= part_rows
                assert sum(len(range(b, T, blocks)) for b in range(blocks)) == T
                continue
            row_vectors(tpr, nv, d, kn)
            block = max(tpr, 512)
            slots = block // tpr
            assert block % tpr == 0 and slots >= 1
            n = min(-(-T // slots), limit)
            assert n <= part_rows
            first = np.arange(n)[:, None] * slots + np.arange(slots)[None]
            hit = np.zeros(T, np.int64)
            for turn in range(-(-T // (n * slots))):
                t = first + turn * n * slots
                np.add.at(hit, t[t < T], 1)
            assert (hit == 1).all()
            if slots > 1:  # the slots' sums meet in an LDS array of nv * tpr * kn floats
                i = np.arange(d)
                vec = i // kn
                at = (vec // tpr * kn + i % kn) * tpr + vec % tpr
                assert at.max() < nv * tpr * kn and np.unique(at).size == d
    assert lib.rmsnorm_bwd_workspace_bytes(0, 64) == 0


# ---- packing (w4_quant.hip) ---------------------------------------------------------
@pytest.mark.parametrize("N,K,group", [(1, 64, 32), (17, 192, 64), (40, 320, 32), (33, 384, 128), (16, 128, 128)])
def test_packing_addresses(N, K, group):
    nt, kt, kg = -(-N // 16), -(-K // 128), K // group
    words, scales, reads = np.zeros(nt * kt * 256, int), np.zeros(nt * kg * 16, int), np.zeros(N * K, int)
    th = np.arange(256)
    r, c8 = th >> 4, th & 15
    for tile in range(nt * kt):
        n, k = tile // kt * 16 + r, tile % kt * 128 + 8 * c8
        ok = (n < N) & (k < K)
        for j in range(8):
            np.add.at(reads, (n * K + k)[ok] + j, 1)
        np.add.at(words, tile * 256 + 64 * (c8 & 3) + 4 * r + (c8 >> 2), 1)
        owner = ((c8 & (group // 8 - 1)) == 0) & (k < K)
        np.add.at(scales, ((tile // kt * kg + k // group) * 16 + r)[owner], 1)
    assert (words == 1).all() and (scales == 1).all() and (reads == 1).all()


# ---- product (w4_matvec.hip) --------------------------------------------------------
BYTES = {"bf16": 2, "i8": 1}


def weight_loads(chk, tile, at, N, K, group, half, zeros):
    """A wave's loads of tile `tile`, chunk `at`: codes, scales, zero points."""
    nt, kt, kg, gp = -(-N // 16), -(-K // 128), K // group, 128 // group
    lane = np.arange(64)
    l16, g = lane & 15, lane >> 4
    ga = ({1: 0 * g, 2: g >> 1, 4: g}[gp]) * 16 + l16
    if half:
        ga = (g & 1 if gp == 4 else 0 * g) * 16 + l16
    tile = min(tile, nt - 1)
    chk("codes", nt * kt * 1024, tile * kt * 1024, kt * 1024, lane * 16, at * 1024, 16)
    chk("scales", nt * kg * 32, tile * kg * 32, kg * 32, ga * 2, at * gp * 32, 2)
    if zeros:
        chk("zeros", nt * kg * 16, tile * kg * 16, kg * 16, ga, at * gp * 16, 1)


SHAPES = [(64, 1, 32), (64, 17, 64), (192, 40, 64), (128, 33, 128), (960, 100, 32), (1088, 530, 64), (4288, 70, 64),
          (12480, 100, 32), (13056, 64, 128)]


@pytest.mark.parametrize("K,N,group", SHAPES)
@pytest.mark.parametrize("x", BYTES)
def test_few_rows_loads(K, N, group, x):
    chk, b = Checker(), BYTES[x]
    kt, nt, gp = -(-K // 128), -(-N // 16), 128 // group
    lane = np.arange(64)
    l16, g = lane & 15, lane >> 4
    for T in (1, 5, 16):
        for R, W in ((1, 16), (2, 16), (4, 8)):
            groups = -(-nt // R)
            for wg in boundary(groups):
                seen = []
                for wave in range(W):
                    nw = -(-(kt - wave) // W) if kt > wave else 0
                    for i in range(nw):
                        at = wave + W * i
                        seen.append(at)
                        half = gp > 1 and at * 128 + 64 == K
                        for r in range(R):
                            weight_loads(chk, wg * R + r, at, N, K, group, half, True)
                        x_at = (np.minimum(l16, T - 1) * K + 8 * g) * b
                        x0 = at * 128 * b
                        for q in range(4):
                            chk("x", T * K * b, 0, T * K * b, x_at + 32 * (q & 1) * b,
                                x0 + (64 * b if q >= 2 and not half else 0), 8 * b)
                assert sorted(seen) == list(range(kt))
    assert chk.loads


# (TB, R, RW, KW) of the kernels that share x through LDS, and whether d_in may be split
SHARED = [((1, 1, 4, 4), True), ((2, 2, 4, 2), False), ((2, 2, 4, 4), False), ((4, 2, 4, 2), False), ((2, 1, 4, 2), True)]


@pytest.mark.parametrize("K,N,group", SHAPES)
@pytest.mark.parametrize("x", BYTES)
@pytest.mark.parametrize("shape,split", SHARED)
def test_shared_rows_loads(K, N, group, x, shape, split):
    (TB, R, RW, KW), b, NS = shape, BYTES[x], 3
    chk = Checker()
    kt, nt, gp = -(-K // 128), -(-N // 16), 128 // group
    row_bytes, waves = 128 * b, RW * KW
    chunk = 16 * TB * row_bytes
    stage = KW * chunk
    copies = stage // 1024
    per = -(-copies // waves)
    pieces = row_bytes // 16
    copy_rows = 64 // pieces
    lane = np.arange(64)
    half_last = gp > 1 and K & 64
    all_steps = -(-kt // KW)
    # the sums of the chunk waves fit the slots
    assert (KW - 1) * R * TB * 4 * RW * 64 * 4 <= NS * stage
    for T in (17, 70) if TB > 1 else (1, 16):
        for t0 in range(0, T, 16 * TB):
            rows = min(T - t0, 16 * TB)
            for splits in ({1, min(3, all_steps), min(16, all_steps)} if split else {1}):
                part = -(-all_steps // splits)
                splits = -(-all_steps // part)  # none empty
                done = []
                for sp in range(splits):
                    step0 = sp * part
                    steps = min(part, all_steps - step0)
                    assert steps > 0
                    for i in boundary(steps + NS):  # run-ahead loads of the last steps too
                        for c in {(w + waves * j) % copies for w in range(waves) for j in range(per)}:
                            at = min((step0 + i) * KW + c * 1024 // chunk, kt - 1)
                            row = c * copy_rows % (16 * TB) + lane // pieces
                            piece = (lane ^ row) & (pieces - 1)
                            off = np.minimum(row, rows - 1) * K * b + 16 * piece
                            if half_last and at == kt - 1:
                                off = off - ((lane ^ (c * copy_rows + lane // pieces)) & (pieces // 2)) * 16
                            chk("x", T * K * b, t0 * K * b, rows * K * b, off, at * row_bytes, 16)
                            assert c * 1024 + 1024 <= stage
                        for kw in range(KW):
                            at = min((step0 + i) * KW + kw, kt - 1)
                            for tile0 in boundary(-(-nt // (R * RW)) * RW):
                                for r in range(R):
                                    weight_loads(chk, tile0 * R + r, at, N, K, group, half_last and at == kt - 1, True)
                    done += [(step0 + i) * KW + kw for i in range(steps) for kw in range(KW) if (step0 + i) * KW + kw < kt]
                assert sorted(done) == list(range(kt))
    # the copies fill a stage, and an operand read finds its logical piece
    phys = {c * 1024 + 16 * ln for c in range(copies) for ln in range(64)}
    assert len(phys) == stage // 16 and {(w + waves * j) % copies for w in range(waves) for j in range(per)} == set(range(copies))
    for row in range(16 * TB):
        for q in range(4):
            for g in range(4):
                byte = (32 * q + 8 * g) * b
                at = row * row_bytes + 16 * (((byte >> 4) ^ row) & (pieces - 1)) + (byte & 15)
                c, ln = at // 1024, at % 1024 // 16
                assert c * copy_rows % (16 * TB) + ln // pieces == row
                assert ((ln ^ row) & (pieces - 1)) * 16 + (at & 15) == byte
    assert chk.loads


def test_workspace_holds_the_partial_sums(lib):
    """splits x T x d_out floats, as many splits as the launch rule of w4_matvec makes."""
    def splits(T, K, N):
        tiles, chunks = -(-N // 16), -(-K // 128)

        def split(groups, kw):
            steps = -(-chunks // kw)
            s = min(512 // groups, steps // 4, 16)
            return 1 if s < 2 else -(-steps // -(-steps // s))

        if T <= 16:
            return 1 if tiles > 768 or chunks < 96 else split(-(-tiles // 4), 4)
        b32, b64, g8 = -(-T // 32), -(-T // 64), -(-tiles // 8)
        if (T > 32 and g8 * b64 >= 192) or g8 * b32 >= 192:
            return 1
        return split(-(-tiles // 4) * b32, 2)

    rng = np.random.default_rng(1)
    seen = set()
    for _ in range(3000):
        T, K, N = int(2 ** rng.uniform(0, 9)), 64 * int(2 ** rng.uniform(0, 9)), int(2 ** rng.uniform(0, 15))
        s = splits(T, K, N)
        seen.add(s)
        need = lib.w4_matvec_workspace_bytes(T, K, N)
        assert need == (0 if s == 1 else -(-s * T * N * 4 // 256) * 256), (T, K, N)
    assert {1, 2, 16} <= seen
