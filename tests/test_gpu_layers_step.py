"""Whole steps whose gradients the layer operators write: a small model of
token and position embeddings, the norms around a block with its gate, and a
linear layer fed from 8-bit activations, through DPStep.step_layers, against
automatic differentiation in 64 bits.

Tolerance, before any run: rows are binary32 here and the output gradients are
exact in bf16, so an element of a gradient is a sum of at most n T products of
values that are each off by some (D + 60) 2^-24 of their magnitude; with D =
96 and n T = 260 that is below 5e-5 of the sum of magnitudes, and the sum of
magnitudes of n T terms of random sign is about sqrt(n T) = 16 times their
sum.  1e-3 of a tensor's norm covers it; a lost term, scale or weight is of order
one."""
import gc

import pytest
import torch

import gradient_reduce_adam_amd as dp
from gradient_reduce_adam_amd import BlockNorm, driver

pytestmark = pytest.mark.gpu

V, C, D, O = 61, 40, 96, 72
NAMES = ("tokens", "bias", "positions", "post_w", "post_b", "gate", "pre_w", "pre_b", "weight")
SHAPES = dict(tokens=(V, D), bias=(O,), positions=(C, D), weight=(O, D))
NUMEL = tuple(int(torch.Size(SHAPES.get(k, (D,))).numel()) for k in NAMES)
AT = {k: i for i, k in enumerate(NAMES)}
OFF = [sum(NUMEL[:i]) for i in range(len(NUMEL) + 1)]
EPS = 1e-5


class Model:
    """One micro-step's forward and backward for every replica, in the framework's operators."""

    def __init__(self, n, a, T, centered, seed, scale=1.5):
        self.n, self.T, self.scale = n, T, scale
        g = torch.Generator().manual_seed(seed)
        self.stream = torch.cuda.Stream()
        self.d = driver.DPStep(NUMEL, n, a, "bf16", "bf16", max_norm=0.5, stream=self.stream)
        master = torch.randn(self.d.P, generator=g) * 0.3
        for k in ("post_w", "pre_w", "gate"):
            master[OFF[AT[k]]:OFF[AT[k] + 1]] += 1
        self.master0 = master.cuda()
        torch.cuda.synchronize()
        self.d.set_master(lambda ptr: self._fill(ptr))
        self.norms = BlockNorm(post_w=AT["post_w"], post_b=AT["post_b"] if centered else None, gate=AT["gate"],
                               pre_w=AT["pre_w"], pre_b=AT["pre_b"] if centered else None, centered=centered, eps=EPS,
                               residual_scale=0.7)
        self.centered = centered
        self.ids = torch.randint(-1, V, (a, n, T), generator=g).cuda()
        self.pos = (torch.arange(T) % C).cuda()
        self.dout = torch.randn((a, n, T, O), generator=g).bfloat16().cuda()
        pl = self.d.plan
        size = max(pl.embed_workspace(AT["tokens"], D, T), pl.embed_workspace(AT["positions"], D, T),
                   pl.block_norm_workspace(self.norms, D, T), pl.linear_workspace(T, D, O, AT["weight"]))
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        f32 = dict(device="cuda", dtype=torch.float32)
        self.h, self.y, self.s, self.x, self.dh, self.dy, self.dx = (
            [torch.empty((T, D), **f32) for _ in range(n)] for _ in range(7))
        self.codes = [torch.empty((T, D), dtype=torch.uint8, device="cuda") for _ in range(n)]
        self.scales = [torch.empty((T, D // 32), dtype=torch.uint8, device="cuda") for _ in range(n)]
        self.xq = torch.empty((a, n, T, D), **f32)
        self.grad = [torch.zeros(self.d.P, dtype=torch.bfloat16, device="cuda") for _ in range(n)]
        for r in range(n):
            pl.bind("grad", self.grad[r], r)
        torch.cuda.synchronize()

    def _fill(self, ptr):
        self.d.master.copy_(self.master0)

    def tensor(self, flat, k):
        return flat[OFF[AT[k]]:OFF[AT[k] + 1]].view(SHAPES.get(k, (D,)))

    def backward(self, step, k, first, loss_scale):
        pl = self.d.plan
        with torch.cuda.stream(self.stream):
            weight = self.tensor(self.d.param, "weight").float()
            for r in range(self.n):
                pl.embed(AT["tokens"], self.ids[k - 1, r], self.h[r], scale=self.scale)
                pl.embed(AT["positions"], self.pos, self.y[r])
                pl.block_norm(self.norms, self.h[r], self.y[r], self.s[r], self.x[r])
                dp.dpl_pack_activations(self.x[r], self.codes[r], self.scales[r])
                dp.dpl_unpack_activations(self.codes[r], self.scales[r], self.xq[k - 1, r])
                torch.mm(self.dout[k - 1, r].float(), weight, out=self.dx[r])
                # the bias' gradient is exact in 16 bits here, and takes the dense path
                self.tensor(self.grad[r], "bias").copy_(self.dout[k - 1, r, :8].float().sum(0).bfloat16())
            pl.accumulate_linear(AT["weight"], self.dout[k - 1].unbind(0), self.codes, self.scales, first, self.ws)
            pl.accumulate_block_norm(self.norms, self.s, self.y, self.dx, None, self.dh, self.dy, first=first,
                                     workspace=self.ws)
            pl.accumulate_embed(AT["tokens"], self.ids[k - 1].unbind(0), self.dh, first, self.ws, scale=self.scale)
            pl.accumulate_embed(AT["positions"], [self.pos] * self.n, self.dy, first, self.ws)
            pl.accumulate_all_range(first, OFF[AT["bias"]], OFF[AT["bias"] + 1])
            if not self.centered:  # the biases of the norms are not used: no gradient
                for b in ("post_b", "pre_b"):
                    pl.accumulate_all_range(first, OFF[AT[b]], OFF[AT[b] + 1])

    def want(self):
        """The averaged gradient by automatic differentiation in 64 bits."""
        p = self.master0.bfloat16().double()
        total = torch.zeros(self.d.P, dtype=torch.float64, device="cuda")
        for k in range(self.ids.shape[0]):
            for r in range(self.n):
                leaf = p.clone().requires_grad_(True)
                t = {name: self.tensor(leaf, name) for name in NAMES}
                ids = self.ids[k, r]
                h = self.scale * t["tokens"][ids.clamp(min=0)] * (ids >= 0)[:, None]
                y = t["positions"][self.pos]

                def norm(v, w, b):
                    if self.centered:
                        v = v - v.mean(-1, keepdim=True)
                    v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS) * t[w]
                    return v + t[b] if self.centered else v

                s = 0.7 * h + t["gate"] * norm(y, "post_w", "post_b")
                x = norm(s, "pre_w", "pre_b")
                dout = self.dout[k, r].double()
                # the weight sees the 8-bit activations, the activations pass their gradient straight through
                out = x @ t["weight"].detach().t() + self.xq[k, r].double() @ t["weight"].t()
                bias = (t["bias"] * dout[:8].sum(0).bfloat16().double()).sum()
                ((out * dout).sum() + bias).backward()
                total += leaf.grad
        return total / self.n


@pytest.mark.parametrize("n,a,centered", [(1, 1, False), (2, 3, True), (3, 2, False)])
def test_step_against_autodiff(n, a, centered):
    m = Model(n, a, 130, centered, seed=n)
    state = m.d.step_layers(m.backward)
    torch.cuda.synchronize()
    got, want = m.d.gbar.double(), m.want()
    for k in NAMES:
        x, y = m.tensor(got, k), m.tensor(want, k)
        assert (x - y).norm() <= 1e-3 * y.norm(), (k, (x - y).norm().item(), y.norm().item())
    norm = want.norm().item()
    assert state["t"] == 1 and abs(state["norm"] - norm) <= 1e-3 * norm
    # the update that follows is the one of this gradient
    g = got * state["gscale"]
    w = m.master0.double() * (1 - 1e-3 * 0.01) - 1e-3 * g / (g.abs() + 1e-8)
    # lr times the ratio's own error where |g| is near eps, binary32 of m and v, and of w
    tol = 1e-3 * 4 * 2.0 ** -23 + m.master0.double().abs() * 2.0 ** -23 + 1e-9
    assert ((m.d.master.double() - w).abs() <= tol).all()
    m.d.close()


def test_captured_step_replays_like_the_eager_one():
    eager, graph = Model(2, 2, 100, True, seed=9), Model(2, 2, 100, True, seed=9)
    for m in (eager, graph):
        m.d.step_layers(m.backward)
    replay = graph.d.capture_layers(graph.backward)
    for k in range(3):
        fresh = torch.randn(graph.dout.shape, generator=torch.Generator().manual_seed(k)).bfloat16().cuda()
        torch.cuda.synchronize()
        for m in (eager, graph):
            m.dout.copy_(fresh)
        torch.cuda.synchronize()
        replay.replay()
        eager.d.step_layers(eager.backward)
        torch.cuda.synchronize()
        assert torch.equal(eager.d.master, graph.d.master) and torch.equal(eager.d.param, graph.d.param)
    assert graph.d.read_state()["t"] == 4
    eager.d.close()
    graph.d.close()


def test_a_tensor_left_out_is_reported():
    m = Model(1, 1, 20, True, seed=4)

    def partial(step, k, first, scale):
        m.d.plan.accumulate_all_range(first, OFF[AT["bias"]], OFF[AT["bias"] + 1])

    with pytest.raises(dp.DpError) as e:
        m.d.step_layers(partial)
    assert e.value.status == dp.DP_ERR_STATE
    m.d.close()


def test_single_pass_and_partials_refuse():
    for kw in (dict(single_pass=True), dict(partials=True)):
        d = driver.DPStep((1024,), 1, 1, "bf16", "bf16", **kw)
        with pytest.raises(ValueError):
            d.step_layers(lambda *x: None)
        d.close()


def test_a_plan_collected_within_a_capture_leaves_it_whole():
    """The garbage collector destroys a plan that has device memory while another plan's call is captured."""
    V, D, T = 16, 8, 40
    g = torch.Generator().manual_seed(3)
    ids, dy = torch.randint(0, V, (T,), generator=g).cuda(), torch.randn((T, D), generator=g).bfloat16().cuda()

    def make():
        p, acc = dp.Plan((V * D,), 1, "bf16", "bf16"), torch.full((V * D,), -7.0, device="cuda")
        p.bind("acc", acc, 0)
        return p, acc, torch.zeros(p.embed_workspace(0, D, T), dtype=torch.uint8, device="cuda")

    plan, acc, ws = make()
    stream = torch.cuda.Stream()
    gc.collect()
    gc.disable()
    try:
        old, other, other_ws = make()
        old.accumulate_embed(0, [ids], [dy], True, other_ws)
        plan.accumulate_embed(0, [ids], [dy], True, ws)
        torch.cuda.synchronize()
        want = acc.clone()
        handle = old.handle
        old.itself = old  # only the collector can free it
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            del old
            gc.collect()
            assert handle in dp._abandoned
            plan.accumulate_embed(0, [ids], [dy], True, ws)
    finally:
        gc.enable()
    for _ in range(3):
        acc.fill_(-7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(acc, want)
    with dp.Plan((1,), 1):
        assert dp._abandoned == []
