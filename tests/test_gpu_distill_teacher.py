"""A teacher's rows that are broken or hold nothing, in the distillation on the GPU."""
import math

import pytest
import torch

from test_gpu_distill import INF, Case

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.mark.parametrize("T,V,dt", [(5, 3, "f32"), (5, 700, "f32"), (5, 50257, "bf16"), (261, 700, "f16"), (3, 150001, "bf16")])
@pytest.mark.parametrize("tail", [False, True])
def test_nan_reaches_the_loss_and_the_whole_gradient(tail, T, V, dt):
    """One NaN in a teacher's row, or nothing else: the row's probabilities are NaN, and so are its loss and its
    gradient; in a place of padding it counts for nothing."""
    c = Case(T, V, 2 if V == 3 else 6, dt, tail=tail, seed=V, weight=False, labels=False)
    c.ids[:4] = torch.arange(c.K, device="cuda")
    c.teacher[0] = NAN
    c.teacher[1, 1] = NAN
    c.teacher[2, 0], c.ids[2, 0] = NAN, -1
    if tail:  # of what is left of the row
        c.total[2] = torch.logsumexp(c.teacher[2, 1:].double() / c.tau, 0).float() + 0.4
    c.call()
    assert torch.isnan(c.loss[:2]).all() and torch.isnan(c.dlogits[:2]).all()
    assert torch.isfinite(c.loss[2:]).all() and torch.isfinite(c.dlogits[2:]).all()


def test_lists_of_minus_infinity():
    """Without totals such a list is no list.  With them its tokens have the teacher's probability 0, and the remainder is
    all of it: KL = -log(what the student gives to the tokens outside the list)."""
    c = Case(3, 100, 5, "f32", weight=False, labels=False)
    c.teacher[1] = -INF
    c.call()
    assert c.loss[1] == 0 and (c.dlogits[1] == 0).all()
    c = Case(3, 100, 5, "f32", tail=True, weight=False, labels=False, seed=1)
    c.ids[1] = torch.arange(5, device="cuda")
    c.teacher[1] = -INF
    c.call()
    logq = torch.log_softmax(c.logits[1].double().cpu(), 0)
    want = -torch.logsumexp(logq[5:], 0).item()
    assert want > 0.01 and math.isclose(c.loss[1].item(), want, rel_tol=1e-5)
    q = logq.exp()
    grad = torch.where(torch.arange(100) < 5, q, q - q / q[5:].sum())
    assert ((c.dlogits[1].double().cpu() - grad).abs() <= 1e-6).all()
