"""The distillation's remainder where the student gives next to nothing to the tokens outside the list: their
exponentials relative to the row's greatest logit leave binary32 from 87 temperatures below it on, the term itself is the
larger the farther they are.  The definition in 64 bits and the bounds are those of test_gpu_distill: relative to the
greatest logit outside the list a sum over these tokens is off by the same r, and the distance of the two greatest logits
by 4 2^-24 of itself, which the bound of log q' holds many times.  To those bounds comes what an exponential of 0 below
2^-126 takes from the gradient of a token outside the list: it is divided by the sum over these tokens.  Relative to the
row's greatest logit that sum is 2^-64 at least, for below it is taken anew with a term of 1: 2^-126 / 2^-64 = 2^-62 of
the factor scale weight soft tau p', p' <= 1."""
import pytest
import torch

import gradient_reduce_adam_amd as dp
from test_gpu_distill import INF, Case

pytestmark = pytest.mark.gpu


def unlisted(c):
    ids = c.ids.cpu().long()
    there = (ids >= 0) & (ids < c.V)
    listed = torch.zeros((c.T, c.V)).scatter_add_(1, torch.where(there, ids, 0), there.float()) > 0
    return ~listed.cuda()


def sunk(gap, *args, **kw):
    """A case whose logits outside the list lie `gap` temperatures lower than they did."""
    c = Case(*args, tail=True, **kw)
    c.logits.copy_(torch.where(unlisted(c), c.logits.float() - gap * c.tau, c.logits.float()))
    return c


def check(c):
    loss, lb, grad, gb = c.want()
    c.call()
    w = c.weight.double().cpu() if c.weight is not None else torch.ones(c.T, dtype=torch.float64)
    gb = gb + 2.0 ** -62 * abs(c.soft) * c.tau * c.scale * w[:, None]
    err = (c.loss.double().cpu() - loss).abs()
    assert (err <= lb).all(), (err / lb).max().item()
    err = (c.dlogits.double().cpu() - grad).abs()
    assert torch.isfinite(c.dlogits).all() and (err <= gb).all(), (err / gb).max().item()


GAPS = [20, 40, 46, 60, 80, 87, 88, 95, 104, 200, 3000]


@pytest.mark.parametrize("dt,scale", [("f32", 65536.0), ("bf16", 65536.0), ("f16", 256.0)])
@pytest.mark.parametrize("tau", [0.25, 1.0, 2.0])
@pytest.mark.parametrize("gap", GAPS)
def test_gaps(gap, tau, dt, scale):
    """Above and below every border: terms that flush, a sum that does, a quotient that a loss scale overflows."""
    check(sunk(gap, 9, 1000, 12, dt, tau=tau, soft=0.8, hard=0.2, seed=gap, scale=scale))


@pytest.mark.parametrize("gap", [50, 87, 120])
@pytest.mark.parametrize("T,V,dt", [(7, 2, "f32"), (7, 5, "bf16"), (5, 8191, "bf16"), (5, 50257, "f16"), (3, 150001, "bf16"), (3, 70001, "f32"),
                                    (261, 501, "f32"), (261, 12001, "bf16"), (259, 30011, "f16")])
def test_every_way_to_keep_a_row(T, V, dt, gap):
    """Rows of one piece, in registers of 1024, 512 and 256 threads, and read piece by piece; in place, too."""
    c = sunk(gap, T, V, min(9, V // 2), dt, tau=1.0, soft=0.5, hard=0.5, seed=V, scale=16.0)
    check(c)
    grad, loss = c.dlogits.clone(), c.loss.clone()
    c.call(dlogits=c.logits)
    assert torch.equal(c.logits, grad) and torch.equal(c.loss, loss)


@pytest.mark.parametrize("gap", [50, 87, 120])
@pytest.mark.parametrize("V,dt", [(1031, "f32"), (9001, "bf16"), (40009, "f32"), (70001, "f16")])
def test_losses_of_many_rows(V, dt, gap):
    """Without a gradient rows are streamed."""
    c = sunk(gap, 260, V, 9, dt, tau=2.0, soft=0.7, hard=0.3, seed=V)
    loss, lb, _, _ = c.want()
    c.call(grad=False)
    err = (c.loss.double().cpu() - loss).abs()
    assert (err <= lb).all(), (err / lb).max().item()


def test_one_listed_token_far_above_all_others():
    """The definition in closed form: the row (g, 0, .., 0), its first token listed with p = 0.9, has the student's
    q = 1 / (1 + 999 e^-g), so KL = 0.9 log 0.9 + 0.1 (log 0.1 + g - log 999) + log(1 + 999 e^-g)."""
    gaps = torch.tensor([10.0, 50.0, 86.0, 87.0, 88.0, 100.0, 1000.0], dtype=torch.float64)
    T, V = len(gaps), 1000
    logits = torch.zeros((T, V), device="cuda")
    logits[:, 0] = gaps.float().cuda()
    ids = torch.zeros((T, 1), dtype=torch.int64, device="cuda")
    teacher = torch.zeros((T, 1), device="cuda")
    total = -torch.full((T,), 0.9, device="cuda").log()
    loss, grad = torch.zeros(T, device="cuda"), torch.zeros((T, V), device="cuda")
    dp.dpd_distill(dp.Distillation(), logits, teacher, ids, loss, grad, total=total, scale=65536.0)
    p = torch.exp(-total.double().cpu())
    rest = 1 - p
    q0 = 1 / (1 + 999 * torch.exp(-gaps))
    want = p * p.log() + rest * (rest.log() + gaps - torch.log(torch.tensor(999.0, dtype=torch.float64))) - q0.log()
    # p is off by 4 2^-24, so p' is; everything else by some 2^-24 of the terms
    assert ((loss.double().cpu() - want).abs() <= 32 * 2.0 ** -24 * (gaps + 8)).all(), (loss, want)
    first, others = 65536 * (q0 - p), 65536 * (((1 - q0) - rest) / 999)
    assert ((grad[:, 0].double().cpu() - first).abs() <= 65536 * 32 * 2.0 ** -24).all()
    assert ((grad[:, 1:].double().cpu() - others[:, None]).abs() <= 65536 * 32 * 2.0 ** -24).all()


def test_a_gradient_scale_that_the_quotient_would_overflow():
    """scale is any finite binary32 number: (1 - p) / s times 1e30 leaves binary32 from a gap of 20 on."""
    for gap in (15, 20, 25, 40, 60):
        check(sunk(gap, 6, 100, 5, "f32", seed=gap, scale=1e30))


def test_nothing_outside_the_list():
    """A list of the whole vocabulary, and one outside which the student gives nothing at all, have no such term."""
    for dead in (False, True):
        c = Case(4, 64, 40 if dead else 64, "f32", tail=True, seed=2, weight=False, labels=False)
        c.ids.copy_(torch.arange(c.K, device="cuda").expand(4, c.K))
        c.logits[:, c.K:] = -INF
        c.call()
        logq = torch.log_softmax(c.logits.double().cpu(), 1)
        logp = c.teacher.double().cpu() - c.total.double().cpu()[:, None]
        p = logp.exp()
        want = (p * (logp - logq[:, :c.K])).sum(1)
        grad = logq.exp() * p.sum(1, keepdim=True)
        grad[:, :c.K] -= p
        assert ((c.loss.double().cpu() - want).abs() <= 1e-5 * (1 + want.abs())).all()
        assert ((c.dlogits.double().cpu() - grad).abs() <= 1e-5).all() and (c.dlogits[:, c.K:] == 0).all()


def test_infinities_and_nan_outside_the_list():
    c = sunk(100, 4, 300, 6, "f32", seed=3, weight=False, labels=False)
    out = unlisted(c)
    at = [int(out[r].nonzero()[7]) for r in range(4)]
    c.logits[0, at[0]] = float("nan")
    c.logits[1, at[1]] = -INF
    c.call()
    assert torch.isnan(c.loss[0]) and torch.isnan(c.dlogits[0]).any()
    want, lb, grad, gb = (x[1:] for x in c.want())
    assert ((c.loss[1:].double().cpu() - want).abs() <= lb).all() and ((c.dlogits[1:].double().cpu() - grad).abs() <= gb).all()


def test_captured():
    c = sunk(90, 20, 5001, 30, "bf16", tau=2.0, hard=0.5, seed=8)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        c.call()
    out = unlisted(c)
    for gap in (0, 80, 300):  # the same graph on rows that need the second sum and on rows that do not
        x = torch.randn((20, 5001), device="cuda")
        c.logits.copy_(torch.where(out, x - gap * c.tau, x))
        check(c)
        loss, grad = c.loss.clone(), c.dlogits.clone()
        c.loss.zero_()
        c.dlogits.fill_(1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.loss, loss) and torch.equal(c.dlogits, grad), gap
