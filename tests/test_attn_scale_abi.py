"""Scales that the attention refuses.  No GPU needed, no kernel is launched."""
import pytest

from test_attn_abi import INVALID, call_attention, lib  # noqa: F401  (lib: the fixture)


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("scale", [1.7014121e38, 2.4e38, 3.4e38, -1e38, 0.0, 1.1e-38])
def test_scales_that_are_refused(lib, prefill, scale):  # noqa: F811
    """Times log2 e they are not finite in fp32, or not positive normal numbers."""
    assert call_attention(lib, prefill, scale=scale) == INVALID
    assert b"scale" in lib.moe_last_error()
