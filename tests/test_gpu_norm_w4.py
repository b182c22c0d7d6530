"""RMS norm, packed 4-bit weights and their product on the GPU against the float64 oracle.

Tolerances. A stored value is off by at most half a step of its type (bf16 2^-8, fp32
2^-24, relative). Float32 sums of m terms are off by at most m 2^-24 of the sum of the
terms' magnitudes; a row's sum here has at most d / 64 terms in a row of additions and
a tree of at most ten more, and about eight roundings around it: F32(d) below.
"""
import numpy as np
import pytest
import torch

from oracle import norm_w4 as o

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F = torch.bfloat16, torch.float32


def F32(d):
    return (d / 64 + 18) * 2.0 ** -24


@pytest.fixture(scope="module")
def q():
    import qlora_linear_amd as q
    q.library()
    return q


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def make(seed, *shape, dtype=BF, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def add_rounded(x, res):
    return (x.float() + res.float()).to(x.dtype)


# ---- norm ---------------------------------------------------------------------------
NORM = [(1, 1), (3, 7), (1, 64), (5, 100), (2, 1001), (9, 2048), (33, 4096), (2, 5003), (4, 5120), (3, 8192),
        (2, 11008), (1, 28672), (2, 32768), (1, 40000), (2, 33333), (700, 96), (600, 1000), (530, 333)]


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,d", NORM)
def test_rmsnorm_fwd(q, T, d, dtype):
    print("rmsnorm_fwd", T, d, dtype, flush=True)
    x, res, w = make(1, T, d, dtype=dtype), make(2, T, d, dtype=dtype, scale=3.0), make(3, d, dtype=dtype)
    x[T // 2] = 0
    for r in (None, res):
        y, h, rstd = q.rmsnorm_fwd(x.cuda(), w.cuda(), 1e-5, residual=None if r is None else r.cuda())
        want_h = x if r is None else add_rounded(x, r)
        assert torch.equal(h.cpu(), want_h)
        ry, rr = o.rmsnorm(host(want_h), host(w), float(np.float32(1e-5)))
        assert np.all(np.abs(host(rstd) - rr) <= F32(d) * rr)
        assert np.all(np.abs(host(y) - ry) <= (HALF[dtype] + F32(d)) * np.abs(ry) + 1e-38)


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,d", NORM)
def test_rmsnorm_fwd_quant(q, T, d, dtype, fmt):
    print("rmsnorm_fwd_quant", T, d, dtype, fmt, flush=True)
    x, res, w = make(4, T, d, dtype=dtype), make(5, T, d, dtype=dtype, scale=3.0), make(6, d, dtype=dtype)
    for r in (res, None):
        if r is None:
            x[T // 2] = 0  # a padded row: scale 0, levels 0
        kind = torch.float8_e4m3fn if fmt == "e4m3" else torch.int8
        lv, scale, h = q.rmsnorm_fwd_quant(x.cuda(), w.cuda(), 1e-5, residual=None if r is None else r.cuda(), qdtype=kind)
        want_h = x if r is None else add_rounded(x, r)
        assert torch.equal(h.cpu(), want_h) and lv.dtype == kind
        ry, _ = o.rmsnorm(host(want_h), host(w), float(np.float32(1e-5)))
        want = np.abs(ry).max(1) / o.TOP[fmt]
        got, s = host(lv), host(scale)
        assert np.all(np.abs(s - want) <= F32(d) * want)
        v = np.divide(ry, want[:, None], out=np.zeros_like(ry), where=want[:, None] > 0)
        step = 0.5 if fmt == "i8" else np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10)
        # the level is the nearest one of a value that is itself off by float32 roundings
        assert np.all(np.abs(got - v) <= step + 4 * F32(d) * np.abs(v))
        assert np.all(got[want == 0] == 0)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,d", NORM + [(1500, 256), (4099, 64)])
def test_rmsnorm_bwd(q, T, d, dtype):
    print("rmsnorm_bwd", T, d, dtype, flush=True)
    h, w, dy, dh = make(7, T, d, dtype=dtype), make(8, d, dtype=dtype), make(9, T, d, dtype=dtype), make(10, T, d, dtype=dtype)
    _, r64 = o.rmsnorm(host(h), host(w), 1e-5)
    rstd = torch.from_numpy(r64.astype(np.float32))
    r = host(rstd)
    g, n = host(dy) * host(w), host(h) * r[:, None]
    for e in (None, dh):
        dx, dw = q.rmsnorm_bwd(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), dh=None if e is None else e.cuda())
        rx, rw = o.rmsnorm_grad(host(dy), host(h), host(w), r, None if e is None else host(e))
        mag = r[:, None] * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(1, keepdims=True))
        mag = mag + (0 if e is None else np.abs(host(e)))
        assert np.all(np.abs(host(dx) - rx) <= HALF[dtype] * np.abs(rx) + F32(d) * mag)
        # at most T additions a column
        assert np.all(np.abs(host(dw) - rw) <= HALF[dtype] * np.abs(rw) + (T + 8) * 2.0 ** -24 * np.abs(host(dy) * n).sum(0))
    frozen, none = q.rmsnorm_bwd(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), dh=dh.cuda(), need_dw=False)
    assert none is None and torch.equal(frozen, dx)


def test_rmsnorm_bwd_against_differences(q):
    """The gradient against central differences of the forward itself, in float32. A step
    of 2^-4 leaves a term of step^2 / 6 times the third derivative (below 1e-3 here) and
    float32 roundings of the loss, about 2^-24 * 200 / 2^-4 (below 1e-3)."""
    T, d = 2, 96
    x, w, dy = make(11, T, d, dtype=F), make(12, d, dtype=F), make(13, T, d, dtype=F, scale=0.1)

    def loss(x):
        y, _, _ = q.rmsnorm_fwd(x.cuda(), w.cuda(), 1e-5)
        return (y.double().cpu() * dy.double()).sum().item()

    y, h, rstd = q.rmsnorm_fwd(x.cuda(), w.cuda(), 1e-5)
    dx, _ = q.rmsnorm_bwd(dy.cuda(), h, w.cuda(), rstd)
    for t, j in [(0, 0), (0, 17), (1, 95), (1, 50)]:
        e = torch.zeros(T, d)
        e[t, j] = 2.0 ** -4
        assert abs((loss(x + e) - loss(x - e)) / 2.0 ** -3 - dx[t, j].item()) < 2e-3


def test_norm_empty_batch(q):
    x, w = torch.empty(0, 64, dtype=BF, device="cuda"), torch.ones(64, dtype=BF, device="cuda")
    y, h, rstd = q.rmsnorm_fwd(x, w, residual=x)
    assert y.shape == h.shape == (0, 64) and rstd.shape == (0,)
    lv, s, _ = q.rmsnorm_fwd_quant(x, w)
    assert lv.shape == (0, 64) and s.shape == (0,)
    dx, dw = q.rmsnorm_bwd(x, x, w, rstd)
    assert dx.shape == (0, 64) and not dw.any()


def test_rmsnorm_bwd_repeats_bit_for_bit(q):
    h, dy, w = make(14, 2000, 1024).cuda(), make(15, 2000, 1024).cuda(), make(16, 1024).cuda()
    rstd = torch.ones(2000, device="cuda")
    first = q.rmsnorm_bwd(dy, h, w, rstd)
    for _ in range(3):
        again = q.rmsnorm_bwd(dy, h, w, rstd)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ---- packed weight ------------------------------------------------------------------
@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("N,K,group", [(1, 64, 32), (16, 128, 128), (37, 192, 64), (5, 320, 32), (130, 1024, 128),
                                       (48, 4160, 64)])
def test_w4_quantize_bit_exact(q, N, K, group, dtype, zero_points):
    print("w4_quantize", N, K, group, dtype, zero_points, flush=True)
    w = make(20, N, K, dtype=dtype, scale=0.02)
    w[0, :group] = 0
    w[N - 1, -group:] = w[N - 1, -group:].abs() + 0.01  # a group of one sign
    codes, scales, zeros = q.w4_quantize(w.cuda(), group, zero_points)
    c, s, z = o.w4_quantize(host(w).astype(np.float32), group, zero_points)
    pc, ps, pz = o.w4_pack(c, s, z)
    assert np.array_equal(codes.cpu().numpy(), pc)
    assert np.array_equal(scales.float().cpu().numpy(), ps)
    assert (zeros is None) != zero_points and (zeros is None or np.array_equal(zeros.cpu().numpy(), pz))
    values = o.w4_values(c, s, z, group)
    for out in (F, BF):
        back = q.w4_dequantize(codes, scales, zeros, d_out=N, d_in=K, dtype=out)
        assert np.array_equal(host(back), values if out == F else o.to_bf16(values).astype(np.float64))


def packed(seed, N, K, group, zero_points, pow2=False):
    """A packed weight from the oracle: (codes, scales, zeros on the GPU, float64 values)."""
    g = np.random.default_rng(seed)
    c = np.clip(np.rint(g.normal(size=(N, K)) * 2.4 + 8), 0, 15).astype(np.uint8)
    s = (2.0 ** g.integers(-2, 3, size=(N, K // group))) if pow2 else o.to_bf16(0.01 * (1 + g.random((N, K // group))))
    s = s.astype(np.float32)
    z = g.integers(0, 16, size=s.shape).astype(np.uint8) if zero_points else np.full(s.shape, 8, np.uint8)
    pc, ps, pz = o.w4_pack(c, s, z)
    # padding rows and columns may hold anything
    pad = np.ones((pc.shape[0] * 16, pc.shape[1] * 128), np.uint8)
    pad[:N, :K] = 0
    junk, _, _ = o.w4_pack(pad * 13, np.zeros((pad.shape[0], 1), np.float32), np.zeros((pad.shape[0], 1), np.uint8))

    ps = ps.copy()
    if N % 16:
        ps[-1, :, N % 16:] = 3.0
    cuda = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()  # noqa: E731
    return (cuda(pc | junk, torch.uint8), cuda(ps, BF), cuda(pz, torch.uint8) if zero_points else None,
            o.w4_values(c, s, z, group))


XT = {"bf16": BF, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
#       T,   K,    N, group
MV = [(1, 64, 1, 32), (1, 64, 16, 64), (2, 128, 17, 128), (3, 192, 37, 64), (4, 4096, 100, 128), (5, 320, 33, 32),
      (8, 1024, 256, 64), (9, 960, 64, 64), (15, 2048, 48, 32), (16, 512, 300, 128), (17, 1152, 40, 128),
      (31, 448, 65, 32), (33, 256, 20, 64), (48, 1024, 129, 128), (64, 640, 130, 64), (65, 640, 31, 128),
      (130, 192, 40, 64), (1, 28672, 48, 128), (3, 8256, 1040, 64), (16, 8192, 4100, 128), (1, 128, 9000, 32),
      # d_in split across workgroups: uneven last splits, a half-filled last chunk, one tile
      (2, 12480, 100, 64), (16, 13056, 530, 128), (11, 28672, 16, 32), (20, 1024, 40, 32), (40, 4288, 70, 64),
      (64, 8192, 520, 128), (33, 4096, 3200, 128), (70, 1088, 33, 64), (24, 192, 24600, 64),
      # four tiles a workgroup; blocks of 64 rows, the last one short
      (3, 192, 12400, 64), (16, 256, 12500, 128), (200, 128, 6500, 32), (64, 320, 24700, 64)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("T,K,N,group", MV)
def test_w4_matvec_exact_on_integers(q, T, K, N, group, zero_points, kind):
    """x small integers, scales powers of two: every product and every partial sum, in any
    order, is a multiple of 1/4 below 2^22, so the float32 result is exact."""
    print("w4_matvec exact", T, K, N, group, zero_points, kind, flush=True)
    codes, scales, zeros, W = packed(T + K + N, N, K, group, zero_points, pow2=True)
    g = np.random.default_rng(K)
    x = g.integers(-3, 4, size=(T, K)).astype(np.float64)
    assert (np.abs(x) @ (np.abs(W).T + 15 * 4)).max() < 2 ** 22  # (the zero point's share too)
    y = q.w4_matvec(torch.from_numpy(x).float().to(XT[kind]).cuda(), codes, scales, zeros, d_out=N, dtype=F)
    assert np.array_equal(host(y), x @ W.T)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("T,K,N,group", [(17, 1856, 24580, 64), (32, 2176, 24580, 128), (50, 1088, 24580, 32)])
def test_w4_matvec_wide_many_steps(q, T, K, N, group, zero_points, kind):
    """Weights wide enough for one block of rows, d_in of several turns of the ring with a
    last step that lacks chunks or half of one. Exact, as above."""
    print("w4_matvec wide", T, K, N, group, zero_points, kind, flush=True)
    codes, scales, zeros, W = packed(T + K, N, K, group, zero_points, pow2=True)
    x = np.random.default_rng(K).integers(-3, 4, size=(T, K)).astype(np.float64)
    assert (np.abs(x) @ (np.abs(W).T + 15 * 4)).max() < 2 ** 22
    y = q.w4_matvec(torch.from_numpy(x).float().to(XT[kind]).cuda(), codes, scales, zeros, d_out=N, dtype=F)
    assert np.array_equal(host(y), x @ W.T)


@pytest.mark.parametrize("out", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("T,K,N,group", [(1, 4096, 300, 128), (6, 1344, 77, 64), (16, 2048, 96, 32), (64, 4096, 64, 128)])
def test_w4_matvec(q, T, K, N, group, kind, out):
    """Random values with row scales. Float32 roundings: a group's sum runs over products of
    x with codes of 0 to 15, some 4 times larger than the differences to the zero point that
    remain of them, in at most group / 8 additions, and K / group group sums are added up:
    as independent roundings of 2^-24 at most 2^-24 (4 sqrt(16) + sqrt(128) + 4), 2^-19 of
    the output's norm."""
    print("w4_matvec", T, K, N, group, kind, out, flush=True)
    codes, scales, zeros, W = packed(K + T, N, K, group, True)
    x = make(30, T, K, dtype=F)
    scale = None
    if kind == "bf16":
        x = x.to(BF)
    else:
        scale = x.abs().amax(1) / (448 if kind == "e4m3" else 127)
        x = x / scale[:, None]
        x = (x.clamp(-448, 448) if kind == "e4m3" else x.round()).to(XT[kind])
    ref = host(x) * (1 if scale is None else host(scale)[:, None]) @ W.T
    y = host(q.w4_matvec(x.cuda(), codes, scales, zeros, d_out=N, x_scale=None if scale is None else scale.cuda(), dtype=out))
    err = np.maximum(np.abs(y - ref) - HALF[out] * np.abs(ref), 0)
    assert np.linalg.norm(err) <= 2.0 ** -19 * np.linalg.norm(ref)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("T", [1, 7, 40])
def test_w4_matvec_multi_equals_single(q, T, kind):
    print("w4_matvec_multi", T, kind, flush=True)
    K, widths = 1024, (256, 40, 1, 129)
    ws = [packed(50 + n, n, K, 64, True) for n in widths]
    x = torch.from_numpy(np.random.default_rng(5).integers(-3, 4, size=(T, K))).float().to(XT[kind]).cuda()
    scale = torch.rand(T, device="cuda")
    ys = q.w4_matvec_multi(x, [w[0] for w in ws], [w[1] for w in ws], [w[2] for w in ws], d_out=widths, x_scale=scale)
    for w, n, y in zip(ws, widths, ys):
        assert torch.equal(y, q.w4_matvec(x, *w[:3], d_out=n, x_scale=scale)) and y.shape == (T, n)


def test_w4_matvec_repeats_and_takes_a_workspace(q):
    """d_in split across workgroups: the same bits each time, on the caller's workspace or not,
    and from two streams at once (a workspace each)."""
    T, K, N = 5, 16384, 200
    codes, scales, zeros, _ = packed(62, N, K, 64, True)
    x = make(34, T, K).cuda()
    need = q.w4_matvec_workspace_bytes(T, K, N)
    assert need > 0
    want = q.w4_matvec(x, codes, scales, zeros, d_out=N, dtype=F)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(q.w4_matvec(x, codes, scales, zeros, d_out=N, dtype=F, workspace=ws), want)
    with pytest.raises(q.LoraNF4Error):
        q.w4_matvec(x, codes, scales, zeros, d_out=N, dtype=F, workspace=ws[:need - 256])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            got.append(q.w4_matvec(x, codes, scales, zeros, d_out=N, dtype=F))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_two_graphs_share_a_workspace(q):
    T, K, N = 3, 16384, 130
    need = q.w4_matvec_workspace_bytes(T, K, N)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    sides = []
    for seed in (63, 64):
        p = packed(seed, N, K, 128, False)
        x = make(seed, T, K).cuda()
        run = lambda p=p, x=x: q.w4_matvec(x, p[0], p[1], d_out=N, dtype=F, workspace=ws)  # noqa: E731
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        sides.append((graph, out, run, x))
    for i in range(4):
        for graph, out, run, x in sides:
            x.copy_(make(100 + i, T, K))
            graph.replay()
        torch.cuda.synchronize()
        for graph, out, run, x in sides:
            assert torch.equal(out, run())


def test_w4_matvec_guard_bands(q):
    """Stores stay inside y for ragged row and token counts."""
    from tests.gpu_util import Guarded
    for T, N in [(1, 1), (5, 33), (17, 100), (64, 15)]:
        codes, scales, zeros, _ = packed(N, N, 256, 64, False)
        x = make(31, T, 256).cuda()
        buf = Guarded(T * N * 2)
        st = q.library().w4_matvec(T, 256, N, 64, 1, x.data_ptr(), None, codes.data_ptr(), scales.data_ptr(), None, 1,
                                   buf.ptr, None, 0, torch.cuda.current_stream().cuda_stream)
        assert st == 0 and buf.canaries_intact()
        assert torch.equal(buf.view(BF, (T, N)), q.w4_matvec(x, codes, scales, zeros, d_out=N))


def test_w4_matvec_infinite_row_stays_in_its_row(q):
    """Rows of x do not mix: an infinity or NaN in one leaves the others as they were."""
    codes, scales, zeros, _ = packed(60, 48, 512, 128, True)
    for T in (4, 20):
        x = make(32, T, 512).cuda()
        want = q.w4_matvec(x, codes, scales, zeros, d_out=48)
        x[1, 5], x[2, 9] = float("inf"), float("nan")
        got = q.w4_matvec(x, codes, scales, zeros, d_out=48)
        keep = [t for t in range(T) if t not in (1, 2)]
        assert torch.equal(got[keep], want[keep]) and not torch.isfinite(got[1:3]).all()


def test_refusals_on_the_binding(q):
    codes, scales, zeros, _ = packed(61, 40, 256, 64, True)
    x = make(33, 2, 256).cuda()
    bad = [lambda: q.w4_matvec(x[:, :128], codes, scales, zeros, d_out=40),
           lambda: q.w4_matvec(x.float(), codes, scales, zeros, d_out=40),
           lambda: q.w4_matvec(x, codes, scales, zeros, d_out=50),
           lambda: q.w4_matvec(x, codes, scales, zeros, d_out=32),
           lambda: q.w4_matvec(x, codes[:, :1].contiguous(), scales, zeros, d_out=40),
           lambda: q.w4_matvec(x, codes, scales.float(), zeros, d_out=40),
           lambda: q.w4_matvec(x, codes, scales, zeros.cpu(), d_out=40),
           lambda: q.w4_matvec(x, codes, scales, zeros, d_out=40, x_scale=torch.ones(3, device="cuda")),
           lambda: q.w4_matvec(x, codes, scales, zeros, d_out=40, dtype=torch.float16),
           lambda: q.w4_matvec_multi(x, [codes], [scales], [None, None]),
           lambda: q.w4_matvec_multi(x, [codes, codes], [scales, scales], [zeros, None]),
           lambda: q.w4_quantize(x, group=16), lambda: q.w4_quantize(x.half()),
           lambda: q.rmsnorm_fwd(x, x[0].float()), lambda: q.rmsnorm_fwd(x.t(), x[0]),
           lambda: q.rmsnorm_fwd(x, x[0], residual=x[:1]), lambda: q.rmsnorm_fwd_quant(x, x[0], qdtype=torch.uint8),
           lambda: q.rmsnorm_bwd(x, x, x[0], torch.ones(3, device="cuda"))]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("not refused:", i)
    with pytest.raises(q.LoraNF4Error):
        q.rmsnorm_fwd(x, x[0], eps=0.0)


# ---- together -----------------------------------------------------------------------
def test_merged_weight_served_in_a_graph(q):
    """Train-side to serve-side: adapters merged, packed, then the norm's 8-bit rows through
    q/k/v, eagerly, on a side stream, and as a captured graph replayed over new inputs."""
    import synth
    from tests.gpu_util import dev_bf16
    K, widths, T = 512, (512, 128, 130), 3
    ws = []
    for i, n in enumerate(widths):
        inp = synth.custom_inputs(70 + i, 1, K, n, 8)
        codes, absmax = q.nf4_quantize(dev_bf16(inp["W"]))
        merged = q.lora_nf4_merge(codes, absmax, dev_bf16(inp["A"]), dev_bf16(inp["B"]), 16.0)
        ws.append((q.w4_quantize(merged, group=64, zero_points=True), merged))
    x, res, w = make(71, T, K).cuda(), make(72, T, K).cuda(), make(73, K).cuda()
    packs = [p for p, _ in ws]

    def step():
        lv, scale, h = q.rmsnorm_fwd_quant(x, w, residual=res)
        return q.w4_matvec_multi(lv, [p[0] for p in packs], [p[1] for p in packs], [p[2] for p in packs], d_out=widths,
                                 x_scale=scale), h

    want, h = step()
    # against the merged weights in float64: 4-bit codes are off by half a step of at most
    # (hi - lo) / 15 (1 + 2^-8), E4M3 rows by 2^-4 of their values
    y64, _ = o.rmsnorm(host(h), host(w), 1e-5)
    for (p, merged), got in zip(ws, want):
        m = host(merged)
        g = m.reshape(m.shape[0], K // 64, 64)
        half = np.repeat((np.maximum(g.max(2), 0) - np.minimum(g.min(2), 0)) / 15 * 0.5 * 1.13, 64, axis=1)
        bound = np.abs(y64) @ half.T + (np.abs(y64) * 2.0 ** -4 + np.abs(y64).max(1, keepdims=True) / 448 * 2.0 ** -10) @ (np.abs(m) + half).T
        assert np.all(np.abs(host(got) - y64 @ m.T) <= bound * 1.01)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other, _ = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(other, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs, hg = step()
    for i in range(4):
        x.copy_(make(80 + i, T, K))
        graph.replay()
        torch.cuda.synchronize()
        want, h = step()
        assert torch.equal(h, hg)
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_training_step_in_a_graph(q):
    """norm -> q/k projections with adapters -> backward -> the norm's gradient, captured and
    replayed: every replay equals the eager step on the same inputs."""
    import synth
    from tests.gpu_util import dev_bf16
    T, K, N, r = 40, 256, 192, 8
    ins = [synth.custom_inputs(90 + i, T, K, N, r) for i in range(2)]
    nf = [q.nf4_quantize(dev_bf16(i["W"])) for i in ins]
    A, B = [dev_bf16(i["A"]) for i in ins], [dev_bf16(i["B"]) for i in ins]
    dys = [dev_bf16(i["dY"]) for i in ins]
    x, res, w, dres = make(91, T, K).cuda(), make(92, T, K).cuda(), make(93, K).cuda(), make(94, T, K).cuda()

    def step():
        y, h, rstd = q.rmsnorm_fwd(x, w, residual=res)
        ys, us = q.lora_nf4_fwd_multi(y, [c for c, _ in nf], [a for _, a in nf], A, B, 16.0)
        dy, dAs, dBs = q.lora_nf4_bwd_multi(y, dys, [c for c, _ in nf], [a for _, a in nf], A, B, 16.0, u_saved=us)
        dx, dw = q.rmsnorm_bwd(dy, h, w, rstd, dh=dres)
        return [*ys, *dAs, *dBs, dx, dw, h]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        x.copy_(make(95 + i, T, K))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b)
