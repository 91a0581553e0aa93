"""Logits up to 2^24 temperatures from 0, where binary32 numbers are one apart, in the distillation on the GPU: rows in
which next to every token but one is out of reach, in the list or outside it.  Definition and bounds of test_gpu_distill
and test_gpu_distill_remainder: a difference of logits is off by 4 2^-24 of itself, which the bounds of log q hold."""
import pytest
import torch

from test_gpu_distill import Case
from test_gpu_distill_remainder import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sigma", [1e3, 6e5])
@pytest.mark.parametrize("tau", [0.25, 1.0, 2.0])
@pytest.mark.parametrize("T,V,dt,tail", [(9, 300, "f32", False), (9, 300, "f32", True), (9, 50257, "bf16", True), (300, 700, "bf16", False),
                                         (300, 3001, "f32", True), (3, 150001, "bf16", True)])
def test_far_logits(T, V, dt, tail, tau, sigma):
    c = Case(T, V, 12, dt, tau=tau, soft=0.7, hard=0.3, tail=tail, seed=V, sigma=sigma)
    assert c.logits.float().abs().max() / min(tau, 1) < 2 ** 24
    check(c)


@pytest.mark.parametrize("sigma", [1e3, 6e5])
def test_far_logits_streamed(sigma):
    c = Case(260, 9001, 12, "bf16", tau=0.5, soft=0.7, hard=0.3, tail=True, seed=1, sigma=sigma)
    loss, lb, _, _ = c.want()
    c.call(grad=False)
    assert ((c.loss.double().cpu() - loss).abs() <= lb).all()
