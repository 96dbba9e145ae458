"""Shapes of the scales of 8-bit rows: in the rows' order, or refused."""
import pytest
import torch

mep = pytest.importorskip("mixture_experts_prefill_amd")


def shaped(*shape, dtype=torch.uint8):
    """Contiguous scales that need no GPU: only their shape is looked at (device index -1)."""
    return mep._scale_args(torch.zeros(shape, dtype=dtype), 6, 128, -1, "x_scale")[1]


@pytest.mark.parametrize("dtype", [torch.uint8, torch.float8_e8m0fnu])
def test_block_scales_of_another_order_are_refused(dtype):
    """4 scales a row, 6 rows: [4, 6] holds as many values, but would be read as other rows' scales."""
    for shape in ((4, 6), (6, 4, 1), (2, 12), (3, 8)):
        with pytest.raises(ValueError, match="x_scale"):
            shaped(*shape, dtype=dtype)
    with pytest.raises(ValueError, match="x_scale"):
        shaped(6, 5, dtype=dtype)
    for shape in ((6, 4), (24,), (2, 3, 4)):
        assert shaped(*shape, dtype=dtype) == mep.SCALE_BLOCK


def test_one_row_and_row_scales_have_one_order():
    assert mep._scale_args(torch.zeros(4, 1, dtype=torch.uint8), 1, 128, -1, "x_scale")[1] == mep.SCALE_BLOCK
    for shape in ((6,), (6, 1), (1, 6)):
        assert shaped(*shape, dtype=torch.float32) == mep.SCALE_ROW
    with pytest.raises(ValueError, match="x_scale"):
        shaped(6, 4, dtype=torch.float32)
