"""The smallest and the largest scale that the attention takes, on the GPU."""
import pytest
import torch

import gradient_reduce_adam_amd as dp
from test_gpu_attention import Case, cut

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,K", [(2, 1), (300, 300), (900, 900)])
def test_smallest_scale(H, K):
    """Every key weighs the same: dv is the mean of what the queries send back, as in the definition."""
    c = Case(cut(100), H, K, 16, "bf16", scale=2.0 ** -100, causal=False, device="cuda")
    c.check()
    assert c.dv.abs().sum() > 0


def test_largest_scale():
    """One key takes all: scores are whole numbers, so none lies next to another."""
    c = Case(cut(64), 2, 1, 64, "bf16", scale=2.0 ** 100, causal=False, device="cuda")
    c.q.copy_(torch.eye(64, device="cuda")[:, None].expand(64, 2, 64))
    c.k.copy_(torch.eye(64, device="cuda")[:, None])
    c.check()
    assert torch.equal(c.out, c.v.expand(64, 2, 64))


@pytest.mark.parametrize("scale", [1.2e-38, 2.0 ** -101, 2.0 ** 101])
def test_refused(scale):
    c = Case(cut(10), 2, 1, 16, "bf16", scale=scale)
    with pytest.raises(dp.DpError, match="scale"):
        c.forward()
    with pytest.raises(dp.DpError, match="scale"):
        c.backward()
    assert (c.out == 3).all() and (c.dk == 3).all()
