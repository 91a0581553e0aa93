"""Whole steps of a small decoder whose forward and backward passes run in the framework's operators from the token ids
to the loss: embedding, norm, 8-bit activations, one projection to queries, keys and values, rotary positions on two
axes in place, attention over packed sequences with grouped keys, an output projection, distillation from a teacher's top
logits beside the labels, and all of it back, through DPStep.step_layers, against automatic differentiation in 64 bits.

Tolerance, before any run: activations and their gradients are stored in f16, a relative step of u = 2^-11 each; a
gradient passes at most 16 stored tensors between the loss and the embedding (logits, their gradient, attention's output
and its gradient, p, ds, q, k, v and their gradients before and after the rotation, the norm's output and input and
theirs), each of which can double the error of what went into it in the norm of a tensor only where terms cancel; 16 times
2 u is 1.6e-2 of a tensor's norm.  The 8-bit inputs of the linear layers enter the reference as stored.  A lost term, mask,
scale or head is of order one."""
import pytest
import torch

import gradient_reduce_adam_amd as dp
from gradient_reduce_adam_amd import BlockNorm, driver

pytestmark = pytest.mark.gpu

V, DIM, H, K, HD, TOP = 211, 96, 6, 2, 32, 12
QKV, OUT = (H + 2 * K) * HD, H * HD
NAMES = ("tokens", "norm", "qkv", "head")
SHAPES = dict(tokens=(V, DIM), norm=(DIM,), qkv=(QKV, DIM), head=(V, OUT))
NUMEL = tuple(int(torch.Size(SHAPES[k]).numel()) for k in NAMES)
AT = {k: i for i, k in enumerate(NAMES)}
OFF = [sum(NUMEL[:i]) for i in range(len(NUMEL) + 1)]
EPS, TAU, SOFT, HARD = 1e-5, 2.0, 0.7, 0.3
SPANS = [(0, 37), (37, 37), (37, 101), (101, 120)]
T = 120


class Model:
    def __init__(self, n, a, window, seed):
        self.n, self.a, self.window = n, a, window
        g = torch.Generator().manual_seed(seed)
        self.stream = torch.cuda.Stream()
        self.d = driver.DPStep(NUMEL, n, a, "f16", "f16", max_norm=0.5, stream=self.stream)
        master = torch.cat([torch.randn(NUMEL[0], generator=g), 1 + 0.2 * torch.randn(NUMEL[1], generator=g),
                            torch.randn(NUMEL[2], generator=g) * 1.5 * DIM ** -0.5, torch.randn(NUMEL[3], generator=g) * OUT ** -0.5])
        self.master0 = master.cuda()
        torch.cuda.synchronize()
        self.d.set_master(lambda ptr: self.d.master.copy_(self.master0))
        self.norms = BlockNorm(pre_w=AT["norm"], eps=EPS)
        self.rotary = dp.Rotary((10, 6), base=100.0)
        self.attention = dp.Attention(causal=True, window=window)
        self.loss_of = dp.Distillation(TAU, SOFT, HARD)
        self.ids = torch.randint(-1, V, (a, n, T), generator=g).cuda()
        self.positions = torch.stack([torch.arange(T) % 37, torch.arange(T) // 7], 1).cuda()
        self.offsets = torch.tensor([0] + [b for _, b in SPANS], dtype=torch.int32).cuda()
        self.teacher = (torch.randn((a, n, T, TOP), generator=g) * 2).half().cuda()
        self.top = torch.stack([torch.randperm(V, generator=g)[:TOP] for _ in range(a * n * T)]).view(a, n, T, TOP).cuda()
        self.labels = torch.randint(-1, V, (a, n, T), generator=g).cuda()
        weight = torch.ones(T)
        weight[5::9] = 0
        self.weight = weight.cuda()
        pl = self.d.plan
        size = max(pl.embed_workspace(AT["tokens"], DIM, T), pl.block_norm_workspace(self.norms, DIM, T),
                   pl.linear_workspace(T, DIM, QKV, AT["qkv"]), pl.linear_workspace(T, OUT, V, AT["head"]),
                   dp.dpa_attention_workspace(T, H))
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        f16 = lambda *s: [torch.zeros(s, dtype=torch.float16, device="cuda") for _ in range(n)]  # noqa: E731
        u8 = lambda *s: [torch.zeros(s, dtype=torch.uint8, device="cuda") for _ in range(n)]  # noqa: E731
        self.zero, self.e, self.s, self.x = torch.zeros((T, DIM), dtype=torch.float16, device="cuda"), f16(T, DIM), f16(T, DIM), f16(T, DIM)
        self.rows, self.drows, self.o, self.do = f16(T, QKV), f16(T, QKV), f16(T, OUT), f16(T, OUT)
        self.logits, self.dx, self.dh = f16(T, V), f16(T, DIM), f16(T, DIM)
        self.lse = [torch.zeros((H, T), device="cuda") for _ in range(n)]
        self.codes, self.scales = u8(T, DIM), u8(T, DIM // 32)
        self.codes2, self.scales2 = u8(T, OUT), u8(T, OUT // 32)
        self.xq, self.oq = torch.zeros((a, n, T, DIM), dtype=torch.float16, device="cuda"), torch.zeros((a, n, T, OUT), dtype=torch.float16, device="cuda")
        self.loss = torch.zeros((a, n, T), device="cuda")
        torch.cuda.synchronize()

    def tensor(self, flat, k):
        return flat[OFF[AT[k]]:OFF[AT[k] + 1]].view(SHAPES[k])

    @staticmethod
    def heads(rows):
        return (rows[:, :H * HD].view(T, H, HD), rows[:, H * HD:(H + K) * HD].view(T, K, HD), rows[:, (H + K) * HD:].view(T, K, HD))

    def backward(self, step, k, first, loss_scale):
        pl, i = self.d.plan, k - 1
        wqkv, whead = self.tensor(self.d.param, "qkv"), self.tensor(self.d.param, "head")
        for r in range(self.n):
            pl.embed(AT["tokens"], self.ids[i, r], self.e[r])
            pl.block_norm(self.norms, self.e[r], self.zero, self.s[r], self.x[r])
            dp.dpl_pack_activations(self.x[r], self.codes[r], self.scales[r])
            dp.dpl_unpack_activations(self.codes[r], self.scales[r], self.xq[i, r])
            torch.mm(self.x[r], wqkv.t(), out=self.rows[r])
            q, kk, v = self.heads(self.rows[r])
            dp.dpa_rotary(self.rotary, self.positions, (q, kk), (q, kk))
            o, do = self.o[r].view(T, H, HD), self.do[r].view(T, H, HD)
            dp.dpa_attention(self.attention, q, kk, v, o, self.lse[r], offsets=self.offsets)
            dp.dpl_pack_activations(self.o[r], self.codes2[r], self.scales2[r])
            dp.dpl_unpack_activations(self.codes2[r], self.scales2[r], self.oq[i, r])
            torch.mm(self.o[r], whead.t(), out=self.logits[r])
            # the gradient takes the logits' place
            dp.dpd_distill(self.loss_of, self.logits[r], self.teacher[i, r], self.top[i, r], self.loss[i, r], self.logits[r],
                           labels=self.labels[i, r], weight=self.weight, scale=loss_scale)
            torch.mm(self.logits[r], whead, out=self.do[r])
            dq, dk, dv = self.heads(self.drows[r])
            dp.dpa_attention_backward(self.attention, q, kk, v, o, self.lse[r], do, dq, dk, dv, self.ws, offsets=self.offsets)
            dp.dpa_rotary(self.rotary, self.positions, (dq, dk), (dq, dk), inverse=True)
            torch.mm(self.drows[r], wqkv, out=self.dx[r])
        pl.accumulate_linear(AT["head"], self.logits, self.codes2, self.scales2, first, self.ws)
        pl.accumulate_linear(AT["qkv"], self.drows, self.codes, self.scales, first, self.ws)
        pl.accumulate_block_norm(self.norms, self.s, None, self.dx, None, self.dh, None, first=first, workspace=self.ws)
        pl.accumulate_embed(AT["tokens"], self.ids[i].unbind(0), self.dh, first, self.ws)

    def want(self):
        """(the averaged gradient, the losses) by automatic differentiation in 64 bits."""
        p = self.master0.half().double()
        total, losses = torch.zeros_like(p), torch.zeros((self.a, self.n, T), dtype=torch.float64, device="cuda")
        for i in range(self.a):
            for r in range(self.n):
                leaf = p.clone().requires_grad_(True)
                w = {k: self.tensor(leaf, k) for k in NAMES}
                ids = self.ids[i, r]
                e = w["tokens"][ids.clamp(min=0)] * (ids >= 0)[:, None]
                x = e / torch.sqrt((e * e).mean(1, keepdim=True) + EPS) * w["norm"]

                def linear(x, stored, weight):
                    # the activations pass through, the weight sees what was stored in 8 bits
                    y = x @ weight.detach().t()
                    through = stored.double() @ weight.t()
                    return y + through - through.detach()

                rows = linear(x, self.xq[i, r], w["qkv"])
                q, kk, v = self.heads(rows)
                j = torch.arange(16, device="cuda")
                angle = self.positions[:, (j >= 10).long()].double() * 100.0 ** (-j.double() / 16)
                c, s = angle.cos()[:, None], angle.sin()[:, None]
                q, kk = (torch.cat([y[..., :16] * c - y[..., 16:] * s, y[..., :16] * s + y[..., 16:] * c], -1) for y in (q, kk))
                o = []
                for a, b in SPANS:
                    back = torch.arange(b - a, device="cuda")[:, None] - torch.arange(b - a, device="cuda")
                    hidden = (back < 0) | (back >= self.window if self.window else back < 0)
                    heads = [torch.softmax((q[a:b, h] @ kk[a:b, h // 3].t() * HD ** -0.5).masked_fill(hidden, -float("inf")), 1) @
                             v[a:b, h // 3] for h in range(H)]
                    o.append(torch.stack(heads, 1))
                z = linear(torch.cat(o).reshape(T, OUT), self.oq[i, r], w["head"])
                pt = torch.softmax(self.teacher[i, r].double() / TAU, 1)
                logq = torch.log_softmax(z / TAU, 1).gather(1, self.top[i, r])
                y = self.labels[i, r]
                ce = -torch.log_softmax(z, 1).gather(1, y.clamp(min=0)[:, None])[:, 0] * (y >= 0)
                loss = SOFT * TAU ** 2 * (pt * (pt.log() - logq)).sum(1) + HARD * ce
                loss = loss * (self.weight > 0)
                losses[i, r] = loss.detach()
                (loss * self.weight).sum().backward()
                total += leaf.grad
        return total / self.n, losses


@pytest.mark.parametrize("n,a,window", [(1, 1, 0), (2, 2, 0), (3, 1, 20)])
def test_step_against_autodiff(n, a, window):
    m = Model(n, a, window, seed=n)
    state = m.d.step_layers(m.backward)
    torch.cuda.synchronize()
    got = m.d.gbar.double()
    want, losses = m.want()
    for k in NAMES:
        x, y = m.tensor(got, k), m.tensor(want, k)
        assert (x - y).norm() <= 1.6e-2 * y.norm(), (k, (x - y).norm().item(), y.norm().item())
    assert (m.loss.double() - losses).norm() <= 1.6e-2 * losses.norm()
    assert state["t"] == 1 and abs(state["norm"] - want.norm().item()) <= 1.6e-2 * want.norm().item()
    m.d.close()


def test_captured_step_replays_like_the_eager_one():
    eager, graph = Model(2, 2, 30, seed=9), Model(2, 2, 30, seed=9)
    for m in (eager, graph):
        m.d.step_layers(m.backward)
    replay = graph.d.capture_layers(graph.backward)
    for k in range(3):
        fresh = torch.randint(-1, V, eager.ids.shape, generator=torch.Generator().manual_seed(k)).cuda()
        torch.cuda.synchronize()
        for m in (eager, graph):
            m.ids.copy_(fresh)
        torch.cuda.synchronize()
        replay.replay()
        eager.d.step_layers(eager.backward)
        torch.cuda.synchronize()
        assert torch.equal(eager.d.master, graph.d.master) and torch.equal(eager.loss, graph.loss)
    assert graph.d.read_state()["t"] == 4
    eager.d.close()
    graph.d.close()
