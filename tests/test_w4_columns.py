"""The width of a packed 4-bit weight from its shapes (CPU)."""
import pytest
import torch

from qlora_linear_amd import norm_w4


def shapes(N, K, group):
    nt = (N + 15) // 16
    return torch.empty(nt, (K + 127) // 128, 1024, dtype=torch.uint8), torch.empty(nt, K // group, 16, dtype=torch.bfloat16)


@pytest.mark.parametrize("K,group", [(k, g) for g in (32, 64, 128) for k in range(64, 1025, 64) if k % g == 0])
def test_columns(K, group):
    assert norm_w4._columns(*shapes(20, K, group), group) == K
    if (K, group) in ((64, 32), (128, 64), (64, 64), (128, 128)):  # the same shapes in pairs
        with pytest.raises(ValueError, match="64 or 128 columns"):
            norm_w4._columns(*shapes(20, K, group), None)
    else:
        assert norm_w4._columns(*shapes(20, K, group), None) == K


def test_columns_refusals():
    codes, scales = shapes(16, 192, 64)
    for bad in (lambda: norm_w4._columns(codes, scales, 32), lambda: norm_w4._columns(codes, torch.empty(1, 5, 16), None),
                lambda: norm_w4._columns(codes, scales[:, :0], None), lambda: norm_w4._columns(codes, None, None),
                lambda: norm_w4._columns(codes[:, :0], scales, None), lambda: norm_w4._columns(codes, scales[0], None)):
        with pytest.raises(ValueError):
            bad()
