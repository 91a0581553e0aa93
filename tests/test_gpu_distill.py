"""The distillation loss and its gradient on the GPU against the formula in 64 bits, and its gradient against
differentiating that formula.

Bounds (e = 2^-24; x: the row's logits below their greatest, over the temperature).  An exponential exp2((z - max) c)
is off by 3 e |x| + 4 e of it; a sum of n by n e besides; so q is off by r = e (4 max|x| over terms that count + V + 12)
relative to it.  Terms with |x| > 110 vanish, so max|x| <= 110, and sums over a thread's, a wave's and a workgroup's
terms have at most V / 256 + 80 additions in a row.  p: the same with the teacher's values; from totals y - total is
rounded, e (|y| + |total|).  The loss sums top terms of p |t - u| and logarithms: 2 (r + top e) of the sum of magnitudes.
The remainder 1 - sum p is off by (top + 8) e + the p's.  The gradient is scale weight times soft tau (q mass - p) and
hard (softmax - 1): r of each term's magnitude, rounded to the type by half a step.  A binary32 exponential gives 0
below the smallest normal number, 2^-126, and divided by a sum of at least 1 it is off by no more: 2 2^-126 (soft tau
+ hard) of the gradient."""
import pytest
import torch

import gradient_reduce_adam_amd as dp

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -126, "f16": 2.0 ** -25, "f32": 2.0 ** -126}
E = 2.0 ** -24
INF = float("inf")


class Case:
    def __init__(self, T, V, K, dt="bf16", tau=1.0, soft=1.0, hard=0.0, tail=False, labels=True, seed=0, ids64=True,
                 teacher_dt=None, pad=0, sigma=2.0, twice=False, weight=True, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.T, self.V, self.K, self.dt, self.tau, self.soft, self.hard, self.scale = T, V, K, dt, tau, soft, hard, scale
        idt = torch.int64 if ids64 else torch.int32
        def padded(x, fill):
            buf = torch.full((x.shape[0], x.shape[1] + pad), fill, dtype=x.dtype, device="cuda")
            view = buf[:, :x.shape[1]]
            view.copy_(x)
            return view

        self.logits = padded((torch.randn((T, V), generator=g) * sigma).to(DT[dt]), float("nan"))
        self.teacher = padded((torch.randn((T, K), generator=g) * 2 + 3).to(DT[teacher_dt or dt]), float("nan"))
        if twice:
            ids = torch.randint(0, max(1, min(V, K // 2)), (T, K), generator=g)
        else:
            ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(T)]) if T and K <= V else torch.zeros((T, K))
        if K > 2:
            ids[::3, -1] = -1
            ids[1::3, 0] = V
        self.ids = padded(ids.to(idt), 0)
        y = torch.randint(0, V, (T,), generator=g)
        if K:
            y[::2] = ids[::2, K // 2]
        y[3::5] = -100
        self.labels = y.to(idt).cuda() if labels else None
        self.total = None
        if tail:
            lists = torch.where((ids >= 0) & (ids < V), self.teacher.cpu().double() / tau, -INF)
            whole = torch.logsumexp(lists, 1) if K else torch.zeros(T, dtype=torch.float64)
            self.total = (torch.where(whole == -INF, torch.zeros_like(whole), whole) + 0.4).float().cuda()
        self.weight = None
        if weight:
            w = torch.rand((T,), generator=g) + 0.5
            w[4::7] = 0
            self.weight = w.cuda()
        self.loss = torch.full((T,), 7.0, device="cuda")
        self.dlogits = padded(torch.full((T, V), 3.0).to(DT[dt]), 5.0)

    def call(self, loss=True, grad=True, dlogits=None):
        dp.dpd_distill(dp.Distillation(self.tau, self.soft, self.hard), self.logits, self.teacher, self.ids,
                       self.loss if loss else None, (self.dlogits if dlogits is None else dlogits) if grad else None,
                       total=self.total, labels=self.labels, weight=self.weight, scale=self.scale)

    def want(self):
        """(loss, its bound, gradient, its bound)."""
        V, K, tau, T = self.V, self.K, self.tau, self.T
        z = self.logits.double().cpu().requires_grad_(True)
        ids = self.ids.cpu().long()
        there = (ids >= 0) & (ids < V)
        at = torch.where(there, ids, 0)
        t = torch.where(there, self.teacher.double().cpu() / tau, -INF)
        if K == 0:
            t, there, at = torch.full((T, 1), -INF, dtype=torch.float64), torch.zeros((T, 1), dtype=torch.bool), torch.zeros((T, 1), dtype=torch.int64)
        own = torch.logsumexp(t, 1, keepdim=True)
        base = self.total.double().cpu()[:, None] if self.total is not None else torch.where(own == -INF, 0.0, own)
        logp = torch.where(there, t - base, 0.0)
        p = torch.where(there, torch.exp(logp), 0.0)
        logq = torch.log_softmax(z / tau, 1)
        kl = torch.where(there, p * (logp - logq.gather(1, at)), 0.0).sum(1)
        sizes = (p * (logp.abs() + logq.detach().gather(1, at).abs())).sum(1) + logq.detach().abs().amin(1)
        rest = torch.zeros(T, dtype=torch.float64)
        rest_off = torch.zeros(T, dtype=torch.float64)
        share = torch.zeros((T, V), dtype=torch.float64)
        if self.total is not None:
            listed = torch.zeros((T, V)).scatter_add_(1, at, there.float()) > 0
            rest = (1 - p.sum(1)).clamp(min=0)
            out = torch.logsumexp(torch.where(listed, -INF, logq), 1)
            some = (rest > 0) & (out != -INF)
            term = rest * (rest.clamp(min=1e-300).log() - torch.where(some, out, 0.0))
            kl = kl + torch.where(some, term, 0.0)
            sizes = sizes + torch.where(some, term.detach().abs(), 0.0)
            rest_off = (K + 8 + 2 * (torch.where(there, t, 0.0).abs().max().item() + base.abs().max().item())) * E * torch.ones(T) * 4
            sizes = sizes + torch.where(some, rest_off * (rest.clamp(min=1e-30).log().abs() + out.detach().abs() + 1) / (64 * E), 0.0)
            share = torch.where(listed | ~some[:, None], 0.0, torch.exp(logq.detach() - out.detach()[:, None]))
        loss = self.soft * tau ** 2 * kl
        mags = abs(self.soft) * tau ** 2 * sizes
        ce_prob = torch.zeros((T, V), dtype=torch.float64)
        if self.hard and self.labels is not None:
            y = self.labels.cpu().long()
            ok = (y >= 0) & (y < V)
            ce = -torch.log_softmax(z, 1).gather(1, y.clamp(0, V - 1)[:, None])[:, 0]
            loss = loss + self.hard * torch.where(ok, ce, 0.0)
            mags = mags + abs(self.hard) * (ce.detach().abs() + z.detach().abs().amax(1))
            ce_prob = torch.where(ok[:, None], torch.softmax(z.detach(), 1) + torch.zeros((T, V), dtype=torch.float64).scatter_(
                1, y.clamp(0, V - 1)[:, None], 1.0), 0.0)
        w = self.weight.double().cpu() if self.weight is not None else torch.ones(T, dtype=torch.float64)
        loss = torch.where(w != 0, loss, 0.0)
        grad = torch.autograd.grad(loss, z, w * self.scale)[0]
        r = (4 * 110 + V / 256 + 100 + K + 2 * (1 + base.abs().max().item())) * E
        spread = torch.zeros((T, V), dtype=torch.float64).scatter_add_(1, at, p)
        gm = abs(self.soft) * tau * (torch.exp(logq.detach()) + spread + rest[:, None] * share) + abs(self.hard) * ce_prob
        gb = 2 * r * gm + 2.0 ** -125 * (abs(self.soft) * tau + abs(self.hard)) + abs(self.soft) * tau * rest_off[:, None] * (share + torch.exp(logq.detach()))
        gb = (gb * (w * self.scale).abs()[:, None]) + U[self.dt] * grad.abs() + TINY[self.dt]
        return loss.detach(), 4 * r * mags + 1e-7 * (1 + loss.detach().abs()), grad, gb

    def check(self, **kw):
        loss, lb, grad, gb = self.want()
        self.call(**kw)
        err = (self.loss.double().cpu() - loss).abs()
        assert (err <= lb).all(), (err / lb).max().item()
        err = (self.dlogits.double().cpu() - grad).abs()
        assert torch.isfinite(self.dlogits).all() and (err <= gb).all(), (err / gb).max().item()
        if self.weight is not None:
            assert (self.loss[4::7] == 0).all() and (self.dlogits[4::7] == 0).all()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V,K", [(1, 1), (2, 1), (7, 3), (8, 8), (9, 4), (100, 10), (1023, 64), (8191, 5), (8193, 20),
                                 (16379, 7), (32761, 30), (50257, 100)])
def test_vocabularies(V, K, dt):
    """One to many pieces a thread; odd sizes put every row at another alignment."""
    Case(9, V, K, dt, tau=2.0, soft=0.7, hard=0.3, seed=V).check()
    Case(9, V, K, dt, tail=V > K, seed=V + 1).check()


@pytest.mark.parametrize("V", [57337, 65537, 106489, 147449, 262144])
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_large_vocabularies(V, dt):
    """Rows that fill the registers, and rows that are read for each pass."""
    Case(3, V, 33, dt, tau=1.5, soft=0.5, hard=0.5, tail=True, seed=V, weight=False).check()


@pytest.mark.parametrize("V,dt", [(500, "f16"), (12001, "bf16"), (12001, "f32"), (30011, "f16"), (50257, "bf16"), (24001, "f32")])
def test_many_rows(V, dt):
    """With more rows than CUs small workgroups take them."""
    Case(261, V, 12, dt, tau=2.0, soft=0.5, hard=0.5, tail=True, seed=V).check()
    c = Case(261, V, 12, dt, tau=0.7, soft=0.5, hard=0.5, seed=V + 1)
    c.call()
    grad = c.dlogits.clone()
    c.call(dlogits=c.logits)
    assert torch.equal(c.logits, grad)


@pytest.mark.parametrize("V,dt", [(1031, "f32"), (9001, "bf16"), (33333, "f32"), (40009, "f32"), (50257, "f16")])
@pytest.mark.parametrize("tau,hard,tail", [(1.0, 0.0, False), (2.0, 0.5, True), (0.7, 0.5, True), (1.0, 1.0, True)])
def test_losses_of_many_rows(V, dt, tau, hard, tail):
    """Without a gradient rows are read once, piece by piece, with sums that follow the greatest logit so far: also
    where it comes last, and behind nothing but -infinity."""
    c = Case(260, V, 9, dt, tau=tau, soft=0.7, hard=hard, tail=tail, seed=V, weight=tail)
    ramp = torch.linspace(-30, 30, V, device="cuda").to(c.logits.dtype)
    c.logits[0], c.logits[1] = ramp, ramp.flip(0)
    c.logits[2, :V - 700] = -INF
    c.ids[2] = torch.arange(V - 9, V, device="cuda").to(c.ids.dtype)
    if c.labels is not None:
        c.labels[2] = V - 3
    loss, lb, _, _ = c.want()
    c.call(grad=False)
    err = (c.loss.double().cpu() - loss).abs()
    assert torch.isfinite(c.loss).all() and (err <= lb).all(), (err / lb).max().item()


@pytest.mark.parametrize("tau", [0.25, 1.0, 2.0, 3.0])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("soft,hard", [(1.0, 0.0), (0.0, 1.0), (0.6, 0.4), (-0.5, 2.0)])
def test_terms(soft, hard, tail, tau):
    Case(11, 501, 17, "f32", tau, soft, hard, tail, seed=3, scale=8.0).check()


@pytest.mark.parametrize("K", [0, 1, 2, 255, 256, 257, 1000, 1024])
@pytest.mark.parametrize("tail", [False, True])
def test_lists(K, tail):
    Case(5, 1500, K, "bf16", hard=0.5, tail=tail, seed=K, ids64=False).check()
    Case(5, 20000, K, "f16", tau=2.0, hard=0.5, tail=tail, seed=K).check()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V,K", [(30, 40), (2000, 300), (40000, 1024)])
def test_tokens_that_occur_twice(V, K, tail):
    """Each occurrence is a term; their probabilities add in the gradient."""
    Case(6, V, K, "f32", tau=2.0, hard=0.2, tail=tail, seed=1, twice=True).check()


def test_a_list_of_the_whole_vocabulary():
    c = Case(4, 64, 64, "f32", tail=True, seed=2)
    c.ids.copy_(torch.arange(64, device="cuda").expand(4, 64))
    c.check()


def test_types_strides_and_no_labels():
    Case(8, 333, 9, "bf16", hard=0.5, pad=3, teacher_dt="f32").check()
    Case(8, 333, 9, "f32", hard=0.5, pad=5, teacher_dt="bf16", ids64=False).check()
    Case(8, 333, 9, "f16", hard=0.5, labels=False, teacher_dt="f16", weight=False, pad=1).check()


def test_lists_of_nothing():
    """Rows whose list is all padding, or holds nothing but -infinity, have no such term."""
    for tail in (False, True):
        c = Case(6, 100, 5, "f32", hard=0.5, tail=tail, weight=False)
        c.ids[0] = -1
        c.check()
    c = Case(6, 100, 5, "f32", soft=1.0, weight=False)
    c.teacher[2] = -INF
    c.call()
    assert c.loss[2] == 0 and (c.dlogits[2] == 0).all()


def test_in_place_and_parts():
    c = Case(10, 5003, 40, "bf16", tau=2.0, hard=0.5, seed=4)
    c.call()
    loss, grad = c.loss.clone(), c.dlogits.clone()
    c.loss.fill_(7)
    c.call(grad=False)
    assert torch.equal(c.loss, loss)
    c.loss.fill_(7)
    c.dlogits.fill_(3)
    c.call(loss=False)
    assert (c.loss == 7).all() and torch.equal(c.dlogits, grad)
    c.call(dlogits=c.logits)
    assert torch.equal(c.loss, loss) and torch.equal(c.logits, grad)


def test_in_place_at_every_alignment_and_size():
    for V in (37, 9000, 33333, 150000):
        c = Case(5, V, 12, "f16", hard=0.5, seed=V, tail=True)
        c.call()
        grad = c.dlogits.clone()
        c.call(dlogits=c.logits)
        assert torch.equal(c.logits, grad), V


def test_steep_and_infinite_logits():
    Case(6, 700, 20, "f32", sigma=40.0, hard=0.5, seed=5).check()
    c = Case(6, 700, 20, "f32", seed=6, weight=False)
    c.logits[0, 5:300] = -INF  # tokens that the student can not give
    keep = torch.arange(300, 320, device="cuda")
    c.ids[0] = keep
    c.check()
    c.logits[1, c.ids[1, 3]] = -INF  # one of the teacher's among them
    c.logits[2, 7] = float("nan")
    c.logits[3, 9] = INF
    c.call()
    assert c.loss[1] == INF and not torch.isnan(c.dlogits[1]).any()
    for r in (2, 3):
        assert torch.isnan(c.loss[r]) and torch.isnan(c.dlogits[r]).any()
    assert torch.isfinite(c.loss[4]) and torch.isfinite(c.dlogits[4]).all()


def test_rows_of_weight_zero_are_not_read():
    c = Case(9, 300, 5, "bf16", hard=0.5, seed=7)
    c.logits[4] = float("nan")
    c.teacher[4] = float("nan")
    c.call()
    assert c.loss[4] == 0 and (c.dlogits[4] == 0).all() and torch.isfinite(c.loss).all()


def test_captured_and_on_streams():
    c = Case(20, 5001, 30, "bf16", tau=2.0, hard=0.5, tail=True, seed=8)
    d = Case(20, 5001, 30, "bf16", tau=2.0, hard=0.5, tail=True, seed=9)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for s, x in ((s1, c), (s2, d)):
        with torch.cuda.stream(s):
            x.call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s1):
        c.call()
    for i in range(3):
        c.logits.copy_(torch.randn((20, 5001), device="cuda").bfloat16())
        c.call()
        torch.cuda.synchronize()
        loss, grad = c.loss.clone(), c.dlogits.clone()
        c.loss.zero_()
        c.dlogits.fill_(i)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.loss, loss) and torch.equal(c.dlogits, grad)


def test_binding_refuses():
    c = Case(6, 50, 4, "bf16")
    D = dp.Distillation()

    def call(d=D, logits=c.logits, teacher=c.teacher, ids=c.ids, loss=c.loss, dlogits=c.dlogits, **kw):
        dp.dpd_distill(d, logits, teacher, ids, loss, dlogits, **kw)

    i32 = c.ids.int()
    for kw in (dict(logits=c.logits.t()), dict(teacher=c.teacher[:5]), dict(ids=c.ids[:, :3]), dict(ids=c.ids.float()),
               dict(loss=c.loss[:5]), dict(loss=c.loss.double()), dict(dlogits=c.dlogits.float()), dict(dlogits=c.dlogits[:, :9]),
               dict(total=c.loss.double()), dict(labels=c.labels.int()), dict(labels=c.labels[:3]), dict(weight=c.loss.half()),
               dict(logits=c.logits.cpu()), dict(ids=c.ids.cpu()), dict(weight=c.loss.cpu()), dict(ids=i32, labels=c.labels),
               dict(logits=c.logits.long())):
        with pytest.raises(ValueError):
            call(**kw)
    wide = torch.zeros((2, 1025), device="cuda")
    for kw in (dict(d=dp.Distillation(temperature=0.0)), dict(d=dp.Distillation(temperature=-1.0)),
               dict(d=dp.Distillation(temperature=float("nan"))), dict(d=dp.Distillation(soft=INF)),
               dict(d=dp.Distillation(hard=float("nan"))), dict(scale=INF), dict(loss=None, dlogits=None),
               dict(dlogits=c.dlogits[:1].expand(6, 50)),
               dict(logits=wide, teacher=wide, ids=wide.long(), loss=None, dlogits=wide)):
        with pytest.raises(dp.DpError):
            call(**kw)
    assert (c.loss == 7).all() and (c.dlogits == 3).all()
    call(logits=c.logits[:0], teacher=c.teacher[:0], ids=c.ids[:0], loss=c.loss[:0], dlogits=c.dlogits[:0])
