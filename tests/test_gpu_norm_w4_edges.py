"""RMS norm and packed 4-bit weights on the GPU where they are easily wrong: scales at a
rounding's border, against the float64 oracle."""
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
