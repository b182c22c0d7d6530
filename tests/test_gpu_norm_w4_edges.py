"""RMS norm and packed 4-bit weights on the GPU where they are easily wrong: scales at a
rounding's border, weights of one tile, rows far from 1, against the float64 oracle."""
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
       "product-overflows": (1e16, 1e23, 1e-5), "rows-far-below-eps": (1e-24, 1e-20, 1e-37)}


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
