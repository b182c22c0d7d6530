"""RMS norm and packed 4-bit weights on the GPU where they are easily wrong: many turns of
the backward's row loop, offsets past 32 bits, scales at a rounding's border, weights of one
tile, rows far from 1, stores between guard bands. Against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import norm_w4 as o

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q():
    import qlora_linear_amd as q
    q.library()
    return q


# ---- packed weight ------------------------------------------------------------------
@pytest.mark.parametrize("zero_points", [False, True])
def test_w4_quantize_scale_next_to_a_tie(q, zero_points):
    """Groups of 64 whose range divided by 7 (15) is next to the middle of two bf16 values:
    scales and codes bit for bit."""
    from tests.test_oracle_w4_scale import near_ties
    r = near_ties(15 if zero_points else 7)
    g = np.random.default_rng(6)
    w = (g.random((r.size, 64), dtype=np.float32) * np.float32(0.9) * r[:, None]).astype(np.float32)
    w[np.arange(r.size), g.integers(0, 64, r.size)] = r
    if not zero_points:
        w[::2] = -w[::2]
    codes, scales, zeros = q.w4_quantize(torch.from_numpy(w).cuda(), 64, zero_points)
    pc, ps, pz = o.w4_pack(*o.w4_quantize(w, 64, zero_points))
    assert np.array_equal(scales.float().cpu().numpy(), ps)
    assert np.array_equal(codes.cpu().numpy(), pc)
    assert not zero_points or np.array_equal(zeros.cpu().numpy(), pz)


@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("K,group", [(64, 32), (64, 64), (128, 64), (128, 128), (128, 32), (192, 64), (320, 32), (960, 64)])
def test_packed_width_by_default(q, K, group, zero_points):
    """Read back without d_in: every column, or an error where 64 and 128 columns have the
    same shapes; never the values of another width."""
    w = torch.randn(20, K, generator=torch.Generator().manual_seed(K)).cuda()
    packed = q.w4_quantize(w, group, zero_points)
    want = q.w4_dequantize(*packed, d_out=20, d_in=K, dtype=F)
    if K // group <= 2 and K <= 128:
        with pytest.raises(ValueError, match="d_in or group"):
            q.w4_dequantize(*packed, d_out=20)
    else:
        assert torch.equal(q.w4_dequantize(*packed, d_out=20, dtype=F), want)
    assert torch.equal(q.w4_dequantize(*packed, d_out=20, dtype=F, group=group), want)
    x = torch.randn(3, K, device="cuda").bfloat16()
    y = q.w4_matvec(x, *packed, d_out=20, dtype=F)
    assert torch.equal(q.w4_matvec(x, *packed, d_out=20, dtype=F, group=group), y)
    lists = [[t] for t in packed[:2]] + ([[packed[2]]] if zero_points else [None])
    assert torch.equal(q.w4_matvec_multi(x, *lists, d_out=[20], dtype=F, group=group)[0], y)
    for wrong in (group * 2, group // 2):
        with pytest.raises(ValueError):
            q.w4_matvec(x, *packed, d_out=20, group=wrong)
    # x of the width that has the same shapes
    other = torch.randn(3, K * 2 if K == 64 else K // 2, device="cuda").bfloat16()
    for call in (lambda: q.w4_matvec(other, *packed, d_out=20, group=group),
                 lambda: q.w4_matvec_multi(other, *lists, d_out=[20], group=group),
                 lambda: q.w4_dequantize(*packed, d_out=20, d_in=other.shape[1], group=group)):
        with pytest.raises(ValueError):
            call()


# ---- norm ---------------------------------------------------------------------------
def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def F32(d):
    """Float32 roundings of a row's statistics and of what is formed from them: a sum of at
    most d / 64 additions in a row and a tree of ten, and eight roundings around it."""
    return (d / 64 + 18) * 2.0 ** -24


# sizes of x's and w's values, and eps
FAR = {"product-underflows": (1e-24, 1e-20, 1e-5), "scale-subnormal": (1.0, 1e-37, 1e-5),
       "scale-of-few-bits": (1.0, 3e-40, 1e-5), "all-below-float32": (1e-30, 1e-25, 1e-5),
       "product-overflows": (1e16, 1e23, 1e-5), "rows-far-below-eps": (1e-24, 1e-20, 1e-37),
       "least-eps": (1e-27, 1e-20, 1.4e-45)}


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("far", FAR)
@pytest.mark.parametrize("T,d", [(4, 48), (3, 1001), (600, 1000), (5, 5003), (3, 33333), (3, 40000)])
def test_rmsnorm_fwd_quant_far_values(q, T, d, far, dtype, fmt):
    """Rows whose h w leaves float32's normal range where h rstd w need not, and scales down to
    a few bits: every level is finite and times its scale the value. y in float32 is off by
    F32(d) of it and half of float32's smallest step, 2^-150; a scale below 2^-126 by one such
    step (it is rounded up), and the levels are those of the scale as it is stored."""
    print("rmsnorm_fwd_quant far", T, d, far, dtype, fmt, flush=True)
    g = torch.Generator().manual_seed(d)
    size, weight, eps = FAR[far]
    x = torch.randn(T, d, generator=g)
    x[0::3] *= size
    x[1::3] = 0
    x, w = x.to(dtype), (torch.randn(d, generator=g) * weight).to(dtype)
    kind = torch.float8_e4m3fn if fmt == "e4m3" else torch.int8
    lv, scale, _ = q.rmsnorm_fwd_quant(x.cuda(), w.cuda(), eps, qdtype=kind)
    y, _ = o.rmsnorm(host(x), host(w), float(np.float32(eps)))
    got, s = host(lv), host(scale)
    top = o.TOP[fmt]
    want = np.abs(y).max(1) / top
    assert np.all(np.abs(s - want) <= F32(d) * want + 1.01 * 2.0 ** -149)
    assert np.all(np.abs(got) <= top) and np.all(s[1::3] == 0)
    zero = s == 0
    assert np.all(got[zero] == 0) and np.all(np.abs(y[zero]) <= 2.0 ** -149)
    v, s = y[~zero] / s[~zero, None], s[~zero, None]
    step = 0.5 if fmt == "i8" else np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10)
    assert np.all(np.abs(got[~zero] - v) <= step + 1.1 * (4 * F32(d) * np.abs(v) + 2.0 ** -150 / s))


HALF = {BF: 2.0 ** -8, F: 2.0 ** -24}


def make(seed, *shape, dtype=BF):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


# More rows than one turn of the backward's workgroups takes, the last turn short: 512
# workgroups of one row at 1024 threads a row, of two at 256, of eight at 64; rows read twice,
# whose dw is summed by 64 workgroups along the rows.
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(5000, 200), (4200, 700), (1100, 2048), (1537, 4096), (600, 5003), (1100, 11008),
                                 (130, 20000), (3, 1 << 20)])
def test_rmsnorm_bwd_many_rows(q, T, d, dtype):
    """Against the oracle, with dh and without, the weight learnt and frozen. A column of dw has
    at most 80 additions one after another here: 10 turns of a thread, 8 rows of a workgroup, 16
    of 512 workgroups and 32 sums of those."""
    print("rmsnorm_bwd", T, d, dtype, flush=True)
    h, w, dy, dh = make(7, T, d, dtype=dtype), make(8, d, dtype=dtype), make(9, T, d, dtype=dtype), make(10, T, d, dtype=dtype)
    rstd = torch.from_numpy(o.rmsnorm(host(h), host(w), 1e-5)[1].astype(np.float32))
    r = host(rstd)[:, None]
    H, W, DY = host(h), host(w), host(dy)
    g, n = DY * W, H * r
    rx, rw = o.rmsnorm_grad(DY, H, W, r[:, 0])
    mag = r * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(1, keepdims=True))
    wide = np.abs(DY * n).sum(0)
    for e in (None, dh):
        dev = [None if t is None else t.cuda() for t in (dy, h, w, rstd, e)]
        dx, dw = q.rmsnorm_bwd(*dev[:4], dh=dev[4])
        E = 0 if e is None else host(e)
        assert np.all(np.abs(host(dx) - rx - E) <= HALF[dtype] * np.abs(rx + E) + F32(d) * (mag + np.abs(E)))
        assert np.all(np.abs(host(dw) - rw) <= HALF[dtype] * np.abs(rw) + 80 * 2.0 ** -24 * wide)
        frozen, none = q.rmsnorm_bwd(*dev[:4], dh=dev[4], need_dw=False)
        assert none is None and torch.equal(frozen, dx)
        again = q.rmsnorm_bwd(*dev[:4], dh=dev[4])
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 1), (3, 7), (5, 1001), (600, 333), (1030, 2047), (2, 5003), (515, 8191), (70, 33333)])
def test_norm_stores_stay_inside(q, T, d, dtype):
    """Every output and the workspace, of exactly their size, between guard bands."""
    from tests.gpu_util import Guarded
    print("norm guards", T, d, dtype, flush=True)
    lib, kind, e = q.library(), 1 if dtype == BF else 0, 2 if dtype == BF else 4
    x, res, w, dh = (make(i, *s, dtype=dtype).cuda() for i, s in enumerate([(T, d), (T, d), (d,), (T, d)]))
    h, y, rstd, lv, sc, dx, dw = (Guarded(n) for n in (T * d * e, T * d * e, T * 4, T * d, T * 4, T * d * e, d * e))
    ws = Guarded(q.rmsnorm_bwd_workspace_bytes(T, d))
    bufs = [h, y, rstd, lv, sc, dx, dw, ws]
    assert lib.rmsnorm_fwd(T, d, kind, 1e-5, x.data_ptr(), res.data_ptr(), w.data_ptr(), h.ptr, y.ptr, rstd.ptr, stream()) == 0
    want = q.rmsnorm_fwd(x, w, 1e-5, residual=res)
    for got, t in zip((y, h, rstd), want):
        assert torch.equal(got.view(t.dtype, t.shape), t)
    for qt, qdtype in ((q.LN_E4M3, torch.float8_e4m3fn), (q.LN_I8, torch.int8)):
        assert lib.rmsnorm_fwd_quant(T, d, kind, 1e-5, x.data_ptr(), res.data_ptr(), w.data_ptr(), h.ptr, qt, lv.ptr,
                                     sc.ptr, stream()) == 0
        a, b, c = q.rmsnorm_fwd_quant(x, w, 1e-5, residual=res, qdtype=qdtype)
        assert torch.equal(lv.view(torch.uint8, (T, d)), a.view(torch.uint8)) and torch.equal(sc.view(F, (T,)), b)
        assert torch.equal(h.view(dtype, (T, d)), c)
    for learnt in (True, False):
        assert lib.rmsnorm_bwd(T, d, kind, x.data_ptr(), dh.data_ptr(), want[1].data_ptr(), w.data_ptr(), want[2].data_ptr(),
                               dx.ptr, dw.ptr if learnt else None, ws.ptr, ws.nbytes, stream()) == 0
        rx, rw = q.rmsnorm_bwd(x, want[1], w, want[2], dh=dh)
        assert torch.equal(dx.view(dtype, (T, d)), rx) and torch.equal(dw.view(dtype, (d,)), rw)
    torch.cuda.synchronize()
    assert all(b.canaries_intact() for b in bufs)


@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("N,K,group", [(1, 64, 32), (17, 192, 64), (40, 320, 32), (33, 384, 128)])
def test_pack_stores_stay_inside(q, N, K, group, zero_points):
    from tests.gpu_util import Guarded
    print("pack guards", N, K, group, flush=True)
    lib = q.library()
    w = make(N, N, K).cuda()
    want = q.w4_quantize(w, group, zero_points)
    codes, scales, zeros, out = (Guarded(n) for n in (want[0].numel(), want[1].numel() * 2, want[1].numel(), N * K * 4))
    z = zeros.ptr if zero_points else None
    assert lib.w4_quantize(w.data_ptr(), 1, N, K, group, codes.ptr, scales.ptr, z, stream()) == 0
    assert lib.w4_dequantize(codes.ptr, scales.ptr, z, N, K, group, 0, out.ptr, stream()) == 0
    torch.cuda.synchronize()
    assert all(b.canaries_intact() for b in (codes, scales, zeros, out))
    for b, t in zip((codes, scales, zeros), want):
        assert t is None or torch.equal(b.view(t.dtype, t.shape), t)
    assert torch.equal(out.view(F, (N, K)), q.w4_dequantize(*want, d_out=N, d_in=K, dtype=F))


# ---- offsets past 32 bits -----------------------------------------------------------
def test_norm_past_32_bits(q):
    """2.15e9 elements, 1025 rows again and again: every block of rows has the first one's bits."""
    n, d, reps = 1025, 4096, 512
    x, w, dy = make(1, n, d).cuda(), make(2, d).cuda(), make(3, n, d).cuda()
    rows = lambda t: t.expand(reps, *t.shape).reshape(-1, *t.shape[1:])  # noqa: E731
    X, DY = rows(x), rows(dy)
    want = q.rmsnorm_fwd(x, w, residual=dy)
    got = q.rmsnorm_fwd(X, w, residual=DY)
    for a, b in zip(got, want):
        assert torch.equal(a, rows(b))
    lv, sc, _ = q.rmsnorm_fwd_quant(X, w)
    a, b, _ = q.rmsnorm_fwd_quant(x, w)
    assert torch.equal(lv.view(torch.uint8), rows(a.view(torch.uint8))) and torch.equal(sc, rows(b))
    dx, dw = q.rmsnorm_bwd(DY, got[1], w, got[2])
    assert torch.equal(dx, rows(q.rmsnorm_bwd(dy, want[1], w, want[2])[0]))
    r = host(want[2])
    terms = host(dy) * host(want[1]) * r[:, None]
    # 513 turns of a thread, two rows of a workgroup, 16 of 512 workgroups and 32 sums of those
    assert np.all(np.abs(host(dw) - reps * terms.sum(0)) <= HALF[BF] * np.abs(reps * terms.sum(0)) +
                  570 * 2.0 ** -24 * reps * np.abs(terms).sum(0))


def test_packing_past_32_bits(q):
    """2.4e9 elements packed and read back: 1024 rows again and again."""
    n, K, reps = 1024, 4096, 576
    w = make(4, n, K).cuda()
    W = w.expand(reps, n, K).reshape(-1, K)
    want = q.w4_quantize(w, 64, True)
    got = q.w4_quantize(W, 64, True)
    for a, b in zip(got, want):
        assert torch.equal(a, b.expand(reps, *b.shape).reshape(a.shape))
    assert torch.equal(q.w4_dequantize(*got, d_in=K), q.w4_dequantize(*want, d_in=K).expand(reps, n, K).reshape(-1, K))


@pytest.mark.parametrize("kind", [BF, torch.int8], ids=["bf16", "i8"])
@pytest.mark.parametrize("T", [3, 20, 64])
def test_w4_matvec_past_32_bits(q, T, kind):
    """4.6e9 bytes of codes: 1024 rows of weight again and again. x small integers, scales
    powers of two: exact in float32 in any order."""
    n, K, group, reps = 1024, 8192, 64, 1100
    g = torch.Generator().manual_seed(T)
    codes = torch.randint(0, 256, (n // 16, K // 128, 1024), generator=g, dtype=torch.uint8).cuda()
    scales = (2.0 ** torch.randint(-2, 3, (n // 16, K // group, 16), generator=g)).to(BF).cuda()
    zeros = torch.randint(0, 16, scales.shape, generator=g, dtype=torch.uint8).cuda()
    x = torch.randint(-1, 2, (T, K), generator=g).to(kind).cuda()
    W = q.w4_dequantize(codes, scales, zeros, d_in=K, dtype=F)
    want = host(x) @ host(W).T
    assert (np.abs(host(x)) @ (np.abs(host(W)).T + 60)).max() < 2 ** 22
    y = q.w4_matvec(x, *(t.expand(reps, *t.shape).reshape(-1, *t.shape[1:]) for t in (codes, scales, zeros)), dtype=F)
    assert np.array_equal(host(y[:, :n]), want)
    assert torch.equal(y, y[:, :n].repeat(1, reps))


def test_w4_matvec_empty_batch(q):
    packed = q.w4_quantize(make(5, 40, 256).cuda(), 64, True)
    x = torch.empty(0, 256, dtype=BF, device="cuda")
    assert q.w4_matvec(x, *packed, d_out=40).shape == (0, 40)
    ys = q.w4_matvec_multi(x, [packed[0]] * 2, [packed[1]] * 2, [packed[2]] * 2, d_out=(40, 33))
    assert [y.shape for y in ys] == [(0, 40), (0, 33)]


# ---- parts of a batch ---------------------------------------------------------------
@pytest.mark.parametrize("rows", [slice(3, 5), slice(1, 7), slice(4, 8), slice(7, 8)])
def test_part_of_a_batch(q, rows):
    """Some rows of a batch with their scales, which need not start on a 16-byte boundary."""
    packed = [q.w4_quantize(make(i, n, 256).cuda(), 64, True) for i, n in enumerate((40, 64))]
    x, w = make(20, 8, 256).cuda(), make(21, 256).cuda()
    lv, scale, _ = q.rmsnorm_fwd_quant(x, w)
    want = q.w4_matvec(lv, *packed[0], d_out=40, x_scale=scale)
    assert torch.equal(q.w4_matvec(lv[rows], *packed[0], d_out=40, x_scale=scale[rows]), want[rows])
    lists = [[p[i] for p in packed] for i in range(3)]
    both = q.w4_matvec_multi(lv, *lists, d_out=(40, 64), x_scale=scale)
    part = q.w4_matvec_multi(lv[rows], *lists, d_out=(40, 64), x_scale=scale[rows])
    assert all(torch.equal(a, b[rows]) for a, b in zip(part, both))
    y, h, rstd = q.rmsnorm_fwd(x, w)
    dx, _ = q.rmsnorm_bwd(y, h, w, rstd)
    assert torch.equal(q.rmsnorm_bwd(y[rows], h[rows], w, rstd[rows])[0], dx[rows])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = q.w4_matvec(lv[rows], *packed[0], d_out=40, x_scale=scale[rows])
    for i in range(4):
        scale.copy_(torch.full_like(scale, 2.0 ** i))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, q.w4_matvec(lv, *packed[0], d_out=40, x_scale=scale)[rows])
    with pytest.raises(ValueError, match="contiguous"):
        q.w4_matvec(lv[:2], *packed[0], d_out=40, x_scale=scale[3:6:2])


# ---- product: several weights in every kernel, the narrowest d_in, many rows ---------
def exact_case(q, seed, T, K, widths, group, zero_points, kind):
    """Packed weights with scales that are powers of two, x of small integers: exact in float32
    in any order of additions. (x, packed weights, float64 products)"""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-2, 3, (T, K), generator=g)
    packs, want = [], []
    for n in widths:
        nt = (n + 15) // 16
        codes = torch.randint(0, 256, (nt, (K + 127) // 128, 1024), generator=g, dtype=torch.uint8).cuda()
        scales = (2.0 ** torch.randint(-2, 2, (nt, K // group, 16), generator=g)).to(BF).cuda()
        zeros = torch.randint(0, 16, scales.shape, generator=g, dtype=torch.uint8).cuda() if zero_points else None
        W = host(q.w4_dequantize(codes, scales, zeros, d_out=n, d_in=K, dtype=F))
        X = x.numpy().astype(np.float64)
        assert (np.abs(X) @ (np.abs(W).T + 30)).max() < 2 ** 22
        packs.append((codes, scales, zeros))
        want.append(X @ W.T)
    return x.float().to(kind).cuda(), packs, want


@pytest.mark.parametrize("kind", [BF, torch.float8_e4m3fn, torch.int8], ids=["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("T,K,widths,group", [
    (5, 16384, (200, 40, 1), 64), (1, 28672, (16, 300), 128),  # d_in split, up to 16 rows
    (20, 4288, (40, 130, 7), 32), (70, 2176, (130, 33), 64),   # d_in split, more rows
    (3, 192, (12300, 50, 17), 32), (16, 256, (3000, 2000), 128),
    (33, 1088, (12000, 5000, 33), 64), (64, 1088, (20000, 4700), 32), (130, 64, (12000, 40), 64)])
def test_w4_matvec_multi_exact(q, T, K, widths, group, zero_points, kind):
    print("w4_matvec_multi exact", T, K, widths, group, zero_points, kind, flush=True)
    x, packs, want = exact_case(q, T + K, T, K, widths, group, zero_points, kind)
    lists = [[p[i] for p in packs] for i in range(3)]
    factor = 2.0 ** torch.randint(-3, 4, (T,), generator=torch.Generator().manual_seed(T)).float()
    for out in (F, BF):
        ys = q.w4_matvec_multi(x, lists[0], lists[1], lists[2] if zero_points else None, d_out=widths,
                               x_scale=factor.cuda(), dtype=out, group=group)
        for y, w in zip(ys, want):
            w = w * host(factor)[:, None]
            assert np.array_equal(host(y), w if out == F else o.to_bf16(w).astype(np.float64))


@pytest.mark.parametrize("kind", [BF, torch.float8_e4m3fn, torch.int8], ids=["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("T,K,N,group", [(1, 64, 40, 64), (20, 64, 40, 32), (64, 64, 24700, 64), (17, 128, 40, 128),
                                         (33, 128, 3100, 32), (1000, 320, 100, 64), (4100, 128, 17, 128)])
def test_w4_matvec_narrow_and_long(q, T, K, N, group, kind):
    print("w4_matvec", T, K, N, group, kind, flush=True)
    x, packs, want = exact_case(q, T + N, T, K, (N,), group, True, kind)
    assert np.array_equal(host(q.w4_matvec(x, *packs[0], d_out=N, dtype=F)), want[0])


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_norm_of_millions_of_rows(q, dtype):
    """More workgroups than lie along one side of a launch."""
    T, d = 4300000, 5
    x, res, w = make(1, T, d, dtype=dtype), make(2, T, d, dtype=dtype), make(3, d, dtype=dtype)
    y, h, rstd = q.rmsnorm_fwd(x.cuda(), w.cuda(), residual=res.cuda())
    assert torch.equal(h.cpu(), (x.float() + res.float()).to(dtype))
    Y, r = o.rmsnorm(host(h), host(w), float(np.float32(1e-5)))
    assert np.all(np.abs(host(rstd) - r) <= F32(d) * r)
    assert np.all(np.abs(host(y) - Y) <= (HALF[dtype] + F32(d)) * np.abs(Y) + 1e-38)
    lv, sc, _ = q.rmsnorm_fwd_quant(x.cuda(), w.cuda(), residual=res.cuda(), qdtype=torch.int8)
    want = np.abs(Y).max(1) / 127
    assert np.all(np.abs(host(sc) - want) <= F32(d) * want)
    assert np.all(np.abs(host(lv) * want[:, None] - Y) <= 0.5 * want[:, None] + 4 * F32(d) * np.abs(Y))
    dx, _ = q.rmsnorm_bwd(x.cuda(), h, w.cuda(), rstd, need_dw=False)
    rx, _ = o.rmsnorm_grad(host(x), host(h), host(w), host(rstd))
    g, n, r = host(x) * host(w), host(h) * host(rstd)[:, None], host(rstd)[:, None]
    mag = r * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(1, keepdims=True))
    assert np.all(np.abs(host(dx) - rx) <= HALF[dtype] * np.abs(rx) + F32(d) * mag)


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("T,d", [(900, 96), (400, 304), (600, 1000), (149, 1992), (36, 6398), (18, 16384), (24, 20660)])
def test_rmsnorm_fwd_quant_halves_go_to_even(q, T, d, fmt):
    """bf16 rows: every level equals the nearest one to the exact quotient v = h w top /
    max |h w|, a quotient in the middle of two levels the even one. h w is A 2^a and the divisor
    M 2^m with A, M < 2^16, a middle k 2^e with k < 2^(b + 1), b <= 7; v / middle is a fraction
    with a numerator or denominator of at most M k or 127 A, so a v that is no middle is
    further from it than 1 / (M k) > 2^-24 2^b / k, half a float32 step: neither float64's
    rounding nor the one to float32 moves it there, and a middle is exact in both."""
    g = torch.Generator().manual_seed(T)
    x, w = make(T, T, d), (1 + 0.2 * torch.randn(d, generator=g)).to(BF)
    kind = torch.float8_e4m3fn if fmt == "e4m3" else torch.int8
    lv, _, _ = q.rmsnorm_fwd_quant(x.cuda(), w.cuda(), qdtype=kind)
    p = host(x) * host(w)
    v = p * o.TOP[fmt] / np.abs(p).max(1, keepdims=True)
    if fmt == "i8":
        halves, want = np.abs(v - np.trunc(v)) == 0.5, np.rint(v)
    else:
        step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)
        halves, want = np.abs(v / step - np.trunc(v / step)) == 0.5, o.e4m3_values()[o.e4m3_encode(v.astype(np.float32))]
    assert halves.any()
    assert np.array_equal(host(lv), want.reshape(T, d))


@pytest.mark.parametrize("kind", [BF, torch.float8_e4m3fn, torch.int8], ids=["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("T", [1, 16, 20, 64])
def test_w4_matvec_widest(q, T, kind):
    """2^22 columns. x is zero but for one column in a thousand and the last ones: sums of at most
    4300 products below 2^7, multiples of 1/4: exact."""
    K, N, group = 1 << 22, 19, 128
    g = torch.Generator().manual_seed(T)
    x = torch.zeros(T, K)
    x[:, ::997] = torch.randint(-1, 2, (T, -(-K // 997)), generator=g).float()
    x[:, -3:] = 1
    codes = torch.randint(0, 256, (2, K // 128, 1024), generator=g, dtype=torch.uint8).cuda()
    scales = (2.0 ** torch.randint(-2, 2, (2, K // group, 16), generator=g)).to(BF).cuda()
    W = q.w4_dequantize(codes, scales, d_out=N, d_in=K, dtype=F)
    on = np.flatnonzero((x != 0).any(0).numpy())
    want = host(x)[:, on] @ host(W)[:, on].T
    y = q.w4_matvec(x.to(kind).cuda(), codes, scales, d_out=N, dtype=F, group=group)
    assert np.array_equal(host(y), want)


@pytest.mark.parametrize("kind", [BF, torch.int8], ids=["bf16", "i8"])
def test_w4_matvec_most_rows(q, kind):
    x, packs, want = exact_case(q, 1, 4096, 64, (17,), 32, True, kind)
    y = q.w4_matvec(x.repeat(512, 1), *packs[0], d_out=17, dtype=F, group=32)
    assert np.array_equal(host(y[:4096]), want[0]) and torch.equal(y, y[:4096].repeat(512, 1))
    with pytest.raises(q.LoraNF4Error):
        q.w4_matvec(x.repeat(513, 1), *packs[0], d_out=17, group=32)


@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("size", [2.0 ** 126, 1e30, 1e-30, 1e-36, 1e-38, 1e-40, 1e-43, 3e-45])
def test_w4_quantize_far_values(q, size, zero_points):
    """float32 weights up to the largest ranges and down to subnormal scales, bit for bit."""
    g = torch.Generator().manual_seed(3)
    w = ((torch.rand(40, 256, generator=g, dtype=torch.float64) * 2 - 1) * size).float()
    w[3, 64:128] = 0
    for group in (32, 128):
        codes, scales, zeros = q.w4_quantize(w.cuda(), group, zero_points)
        c, s, z = o.w4_quantize(w.numpy(), group, zero_points)
        pc, ps, pz = o.w4_pack(c, s, z)
        assert np.array_equal(scales.float().cpu().numpy(), ps)
        assert np.array_equal(codes.cpu().numpy(), pc)
        assert not zero_points or np.array_equal(zeros.cpu().numpy(), pz)
        assert np.array_equal(host(q.w4_dequantize(codes, scales, zeros, d_out=40, d_in=256, dtype=F)),
                              o.w4_values(c, s, z, group).astype(np.float32))
