"""The index arithmetic of kv4_append.hip and kv4_attention.hip restated on the host: every
access inside its operand, every element by one thread, every key tile of a row block by one
worker, every part that is written joined once, and the workspace as large as what is put in it."""
import os
import random

import pytest

DIMS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]


@pytest.fixture(scope="module")
def lib():
    import qlora_linear_amd as q
    if not os.path.exists(q.library_path):
        from qlora_linear_amd import build
        build.build()
    return q.library()


# ---- pages ----------------------------------------------------------------------------
def test_page_of_a_tile():
    """(t * inv) >> 32 with inv = ceil(2^32 / tiles) is t / tiles for every tile of 2^30 keys."""
    for tiles in range(2, 129):
        inv = ((1 << 32) + tiles - 1) // tiles
        most = (1 << 30) // 32
        for t in {0, 1, tiles - 1, tiles, most - 1, most, *(k * tiles + d for k in (7, 1000, most // tiles - 1) for d in (-1, 0, 1))}:
            assert (t * inv) >> 32 == t // tiles, (tiles, t)


@pytest.mark.parametrize("D,G", DIMS)
def test_loads_of_a_tile(D, G):
    """The 64 lanes' codes and scales of a tile, keys and values: inside the tile's rows of its page
    and head, each byte once."""
    for page in (32, 96, 4096):
        for tok in (0, page - 32):
            base = tok * (D // 2)
            keys = [base + s * 16 * (D // 2) + (lane & 15) * (D // 2) + (lane >> 4) * (D // 8) + b
                    for s in range(2) for lane in range(64) for b in range(D // 8)]
            values = [base + s * 8 * D + (lane >> 4) * 2 * D + (lane & 15) * (D // 8) + b
                      for s in range(2) for lane in range(64) for b in range(D // 8)]
            for at in (keys, values):
                assert sorted(at) == list(range(base, base + 32 * (D // 2)))
                assert base + 32 * (D // 2) <= page * (D // 2)
            groups = D // G
            if groups == 1:
                words = [tok + lane % 32 for lane in range(64)]
                assert sorted(words) == sorted(2 * list(range(tok, tok + 32)))
            else:
                words = [(2 * i + lane // 32) * page + tok + lane % 32 for i in range(groups // 2) for lane in range(64)]
                assert sorted(words) == sorted(g * page + tok + k for g in range(groups) for k in range(32))
            assert max(words) < groups * page


# ---- append ---------------------------------------------------------------------------
def append_threads(D, N, chunk, turned):
    pieces, tile = D // 8, 1 if N == 1 else 8 if D == 256 else 16
    heads = 2048 // D if N == 1 else 8 if D == 64 else 4
    for tid in range(256):
        piece, rest = tid % pieces, tid // pieces
        if chunk < turned:
            i, h0 = rest % tile, chunk * heads + rest // tile * N
            for n in range(N):
                yield i, h0 + n, piece, tid
        else:
            h, i0 = (chunk - turned) * heads + rest % heads, rest // heads * N
            for n in range(N):
                yield i0 + n, h, piece, tid


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("N", [1, 4])
def test_append_covers_every_piece(D, N):
    tile = 1 if N == 1 else 8 if D == 256 else 16
    heads = 2048 // D if N == 1 else 8 if D == 64 else 4
    for n_q, n_kv in ((0, 1), (4, 4), (7, 7), (32, 8), (40, 40), (3, 1)):
        turned = (n_q + n_kv + heads - 1) // heads
        for first, count, lo, hi in ((0, turned, 0, n_q + n_kv), (turned, (n_kv + heads - 1) // heads, 0, n_kv)):
            seen = [(i, h, p) for c in range(first, first + count) for i, h, p, _ in append_threads(D, N, c, turned) if h < hi]
            assert len(seen) == len(set(seen)) == tile * hi * (D // 8)
            assert all(0 <= i < tile for i, _, _ in seen)
    # a group's lanes: 4, 8 or 16 neighbours of a row of 16, of one token and head
    for c in range(2):
        lanes = {tid: (i, h, p) for i, h, p, tid in append_threads(D, N, c, 1)}
        for size in (4, 8, 16):
            if size <= D // 8:
                for t0 in range(0, 256, size):
                    assert len({lanes[t][:2] for t in range(t0, t0 + size)}) == 1
                    assert [lanes[t][2] % size for t in range(t0, t0 + size)] == list(range(size))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_stores(D):
    """A token's bytes: a key's row by words, a value's by single bytes or, of four tokens, by words;
    each byte once, none of another token's."""
    keys, single, four = [], [], []
    for piece in range(D // 8):
        d0 = 8 * piece
        chunk, seg = d0 // 32, d0 % 32 // 8
        keys += [seg * (D // 8) + 4 * chunk + b for b in range(4)]
        for j in range(4):
            at = 4 * seg * (D // 8) + 4 * chunk + j * (D // 8)
            single += [(at + tok) for tok in range(4)]
            four += [at + b for b in range(4)]
    assert sorted(keys) == list(range(D // 2)) and sorted(single) == sorted(four) == list(range(2 * D))
    from oracle import kv4 as o
    for piece in range(D // 8):
        d0 = 8 * piece
        chunk, seg = d0 // 32, d0 % 32 // 8
        for j in range(8):  # the word's nibbles
            assert o.k_place(D, d0 + j) == (seg * (D // 8) + 4 * chunk + j % 4, 4 * (j // 4))
            for tok in range(4):
                assert o.v_place(D, d0 + j, tok) == (4 * seg * (D // 8) + 4 * chunk + j // 2 * (D // 8) + tok, 4 * (j % 2))


# ---- shares ---------------------------------------------------------------------------
def most_nq(D, G):
    return (4 if G == 64 else 2) if D == 64 else 2 if D == 128 else 1


def waves(D, G, nq, solo):
    if D == 64:
        return 4 if nq == 1 else 3 if nq == 2 and (solo or G == 64) else 2
    return 3 if D == 128 and nq == 1 else 2


def plan(T, B, n_q, n_kv, D, max_q, max_len, G):
    heads = n_q // n_kv
    most = max_q * heads if max_q else -(-T * heads // B)
    nq = min(1 if most <= 16 else 2 if most <= 32 else 4, most_nq(D, G))
    blocks = -(-most // (16 * nq))
    in_seq = blocks if max_q and B * blocks <= 512 else 0
    items = B * blocks if in_seq else T * heads // (16 * nq) + min(T, B)
    solo = items * n_kv >= 1024
    workers = 256 * waves(D, G, nq, solo) * (4 if solo else 1)
    by_head = in_seq == 1 and items * n_kv < workers
    cuts = items * n_kv if by_head else workers
    whole = in_seq != 0 and not solo and max_len <= 512 and items * n_kv <= workers
    if whole:
        workers, by_head, cuts = items * n_kv, False, 0
    cost = (4 if not solo else 1, *{1: (1, 1, 2), 2: (3, 2, 6), 4: (5, 2, 15)}[nq])
    return dict(nq=nq, in_seq=in_seq, items=items, solo=solo, workers=workers, by_head=by_head, cuts=cuts, whole=whole, cost=cost)


def space(p, B, D):
    up = lambda n: (n + 255) & ~255  # noqa: E731
    rows = 0 if p["whole"] else p["workers"] * 2 * 16 * p["nq"]
    return sum(map(up, (4, B * 4, (p["items"] + 1) * 8, p["items"] * 4, rows * D * 4, rows * 8, p["cuts"] * 32)))


def test_workspace_is_what_the_plan_takes(lib):
    r = random.Random(1)
    for _ in range(400):
        D = r.choice([64, 128, 256])
        n_kv = r.choice([1, 2, 8, 40])
        n_q = n_kv * r.choice([1, 3, 4, 8, 16])
        B = r.choice([1, 2, 17, 96, 511, 512, 513, 3000])
        max_q = r.choice([0, 1, 1, 5, 300])
        T = B if max_q == 1 else r.randint(1, 4 * B)
        page, pages = r.choice([32, 64, 96]), r.choice([1, 5, 16, 17, 4000])
        want = max(space(plan(T, B, n_q, n_kv, D, max_q, pages * page, G), B, D) for G in (32, 64, 128))
        assert lib.kv4_attention_workspace_bytes(T, B, n_q, n_kv, D, max_q, pages, page) == want


def units_of(rows, lo, hi, cost):
    tiles, step, step16, block = cost
    n = -(-(-(-hi // 32) - lo // 32) // tiles)
    return block + n * (step16 if rows <= 16 else step), n


def step_at(x, rows, cost):
    u = cost[2] if rows <= 16 else cost[1]
    return 0 if x <= cost[3] else -(-(x - cost[3]) // u)


@pytest.mark.parametrize("seed", range(60))
def test_shares_and_parts(seed):
    """Row blocks of any rows and keys laid end to end and cut into shares: each step of each
    row block and head in one share, parts in places of their own, and the join of a cut takes
    exactly the workers that have part of it."""
    r = random.Random(seed)
    cost = r.choice([(4, 1, 1, 2), (1, 1, 1, 2), (4, 3, 2, 6), (1, 3, 2, 6), (1, 5, 2, 15)])
    n_kv = r.choice([1, 2, 5])
    most_workers = r.choice([1, 2, 7, 64, 300])
    blocks = []
    for _ in range(r.randint(1, 40)):
        if r.random() < 0.15:
            blocks.append(None)  # a row block that a sequence does not have: no units
        else:
            hi = r.choice([0, 1, 31, 32, 33, 500, r.randint(0, 9000)])
            blocks.append((r.choice([0, 1, 16, 17, 64]), r.randint(0, hi), hi))
    blocks[0] = blocks[0] or (1, 0, 40)
    before = [0]
    for b in blocks:
        before.append(before[-1] + (units_of(*b, cost)[0] if b else 0))
    units = before[-1] * n_kv
    workers = min(most_workers, units)
    share = lambda w: w * units // workers  # noqa: E731
    done, parts, cuts, whole = {}, {}, {}, set()
    for me in range(workers):
        at, end = share(me), share(me + 1)
        assert at < end
        item = max(i for i in range(len(blocks)) if before[i] * n_kv <= at)
        begun = 0
        while at < end:
            own = before[item + 1] - before[item]
            if own == 0:
                item += 1
                continue
            h = (at - before[item] * n_kv) // own
            u0 = at - before[item] * n_kv - h * own
            u1 = min(own, u0 + end - at)
            assert 0 <= h < n_kv and 0 <= u0 < u1
            rows = blocks[item][0]
            for s in range(step_at(u0, rows, cost), step_at(u1, rows, cost)):
                assert (item, h, s) not in done
                done[item, h, s] = me
            if u0 == 0 and u1 == own:
                whole.add((item, h))
            else:
                place = 2 * me + (1 if u0 == 0 else 0)
                assert place not in parts
                parts[place] = (item, h)
            if u0 == 0 and u1 < own:
                begun += 1
                last = ((at + own) * workers - 1) // units
                cuts[item, h] = (me, last)
            at += u1 - u0
            if u1 == own and h == n_kv - 1:
                item += 1
        assert begun <= 1
    for i, b in enumerate(blocks):
        if b is None:
            continue
        n = units_of(*b, cost)[1]
        for h in range(n_kv):
            assert all((i, h, s) in done for s in range(n)) and (i, h, n) not in done
            assert ((i, h) in whole) != ((i, h) in cuts)
            if (i, h) in cuts:
                w0, w1 = cuts[i, h]
                assert w1 > w0
                joined = [2 * w + (1 if w == w0 else 0) for w in range(w0, w1 + 1)]
                assert all(parts[p] == (i, h) for p in joined)
                assert [p for p, v in parts.items() if v == (i, h)] == joined


def test_row_blocks_fit_their_list():
    """Row blocks of sequences whose rows add up to T are no more than the workspace lists."""
    r = random.Random(5)
    for _ in range(300):
        heads, R = r.choice([1, 3, 4, 8, 16, 100]), r.choice([16, 32, 64])
        n = [r.choice([0, 1, 1, 5, r.randint(0, 300)]) for _ in range(r.randint(1, 50))]
        T = sum(n)
        assert sum(-(-m * heads // R) for m in n) <= T * heads // R + min(T, len(n))
