"""Scales of the attention that binary32 has no room for, refused on the host: the backward pass starts its scores at
-lse / scale, which overflows for scales next to the smallest numbers and would leave dk and dv zero."""
import pytest

pytest.importorskip("gradient_reduce_adam_amd")
from test_attention_host import backward, desc, forward, refused  # noqa: E402


@pytest.mark.parametrize("scale", [1.2e-38, 1e-37, 1e-34, 2.0 ** -101, 2.0 ** 101, 1e38])
def test_scales_out_of_range(scale):
    assert "scale" in refused(forward(desc(scale=scale)))
    assert "scale" in refused(backward(desc(scale=scale)))
