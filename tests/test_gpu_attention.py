"""Attention and its backward pass on the GPU against the definition in 64 bits, with the bounds that
attention_common derives: lengths from one, odd heads, grouped keys, windows, rows that see nothing, packed and
padded batches, strides and alignments, streams and captured calls."""
import math

import pytest
import torch

import gradient_reduce_adam_amd as dp
from attention_common import DT, backward, compare, forward, lengths

pytestmark = pytest.mark.gpu


class Case:
    """Inputs of a call and its buffers, which hold a pattern where nothing may be written."""

    def __init__(self, spans, H, K, D, dt, seed=0, spans_k=None, causal=True, window=0, T=None, Tk=None, layout="own",
                 sigma=1.0, scale=None, device="cpu"):
        g = torch.Generator().manual_seed(seed)
        self.spans, self.spans_k = spans, spans_k or spans
        self.T = T or max([b for _, b in spans] + [0])
        self.Tk = Tk or (max([b for _, b in self.spans_k] + [0]) if spans_k else self.T)
        self.H, self.K, self.D, self.dt, self.causal, self.window = H, K, D, dt, causal, window
        self.scale = scale or 1 / math.sqrt(D)
        self.q, self.k, self.v = (self.tensor(t, n, layout, torch.randn((t, n, D), generator=g) * sigma)
                                  for t, n in ((self.T, H), (self.Tk, K), (self.Tk, K)))
        self.dout = self.tensor(self.T, H, layout, torch.randn((self.T, H, D), generator=g) * 0.1)
        self.out, self.dq = (self.tensor(self.T, H, layout, torch.full((self.T, H, D), 3.0)) for _ in range(2))
        self.dk, self.dv = (self.tensor(self.Tk, K, layout, torch.full((self.Tk, K, D), 3.0)) for _ in range(2))
        self.lse = torch.full((H, self.T), 5.0, device="cuda")
        self.ws = torch.empty(max(1, dp.dpa_attention_workspace(self.T, H)), dtype=torch.uint8, device="cuda")
        self.attention, self.device = dp.Attention(causal=causal, window=window, scale=scale), device

    def tensor(self, t, n, layout, x):
        x, D = x.to(DT[self.dt]).cuda(), self.D
        nan = float("nan")
        if layout == "own":
            return x
        if layout == "rows":  # heads side by side in wider rows, at an odd address
            buf = torch.full((t * (n * D + 5) + 1,), nan, dtype=x.dtype, device="cuda")
            view = buf[1:].view(t, n * D + 5)[:, :n * D].view(t, n, D) if t else x
        elif layout == "heads":  # the heads outside, with gaps
            buf = torch.full((n, t * (D + 3)), nan, dtype=x.dtype, device="cuda")
            view = buf.view(n, t, D + 3)[:, :, :D].transpose(0, 1)
        return view.copy_(x)

    def places(self, form="offsets", dtype=torch.int32):
        def of(spans, T):
            if form == "spans":
                return torch.tensor(spans, dtype=dtype).view(-1, 2).cuda()
            return lengths(spans, T).to(dtype).cuda()

        return dict(offsets=of(self.spans, self.T), offsets_k=None if self.spans_k is self.spans else of(self.spans_k, self.Tk))

    def forward(self, **places):
        dp.dpa_attention(self.attention, self.q, self.k, self.v, self.out, self.lse, **places)

    def backward(self, **places):
        dp.dpa_attention_backward(self.attention, self.q, self.k, self.v, self.out, self.lse, self.dout, self.dq, self.dk,
                                  self.dv, self.ws, **places)

    def check(self, **places):
        old = {x: getattr(self, x).clone() for x in ("out", "lse", "dq", "dk", "dv")}
        self.forward(**places)
        args = (self.spans, self.spans_k, self.causal, self.window, self.scale, self.dt, self.device)
        out, lse, eo, el = forward(self.q, self.k, self.v, *args)
        compare("out", self.out, out, eo, old["out"])
        compare("lse", self.lse, lse, el, old["lse"])
        self.backward(**places)
        # from the values that the backward pass read
        grads, bounds = backward(self.q, self.k, self.v, self.out, self.lse, self.dout, *args)
        for name, want, bound in zip(("dq", "dk", "dv"), grads, bounds):
            compare(name, getattr(self, name), want, bound, old[name])


def cut(*ls):
    spans, at = [], 0
    for n in ls:
        spans.append((at, at + n))
        at += n
    return spans


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 257])
def test_lengths(L, dt):
    Case(cut(L), 2, 1, 64, dt, seed=L).check()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [8, 16, 24, 32, 40, 48, 56, 64, 72, 80, 88, 96, 104, 112, 120, 128])
def test_heads_of_every_size(D, causal):
    Case(cut(150), 2, 2, D, "bf16", seed=D, causal=causal).check()


@pytest.mark.parametrize("H,K", [(1, 1), (3, 1), (4, 2), (6, 3), (8, 1), (5, 5)])
def test_heads_that_share_keys(H, K):
    Case(cut(70, 33), H, K, 40, "f16", seed=H).check(**Case(cut(70, 33), H, K, 40, "f16").places())


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("window", [1, 2, 31, 64, 65, 100, 1 << 40])
def test_windows(window, causal):
    Case(cut(190), 2, 1, 32, "bf16", seed=window % 97, causal=causal, window=window).check()


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 20), (False, 20)])
@pytest.mark.parametrize("L,M", [(1, 300), (300, 1), (65, 200), (200, 65), (7, 7), (130, 0), (33, 129)])
def test_other_keys_and_rows_that_see_none(L, M, causal, window):
    """With more queries than keys under a causal mask the first queries see nothing."""
    c = Case(cut(L), 2, 2, 64, "bf16", seed=L + M, spans_k=cut(M) if M else [(0, 0)], Tk=M, causal=causal, window=window)
    c.check(**c.places())
    if causal and L > M:
        assert (c.out[:L - M] == 0).all() and (c.lse[:, :L - M] == -float("inf")).all() and (c.dq[:L - M] == 0).all()


@pytest.mark.parametrize("form,dtype", [("offsets", torch.int32), ("offsets", torch.int64), ("spans", torch.int32),
                                        ("spans", torch.int64)])
@pytest.mark.parametrize("layout", ["own", "rows", "heads"])
def test_packed_batches(layout, form, dtype):
    """Sequences of none to many rows, rows before the first and behind the last one, which stay as they were."""
    spans = [(a + 3, b + 3) for a, b in cut(5, 0, 128, 1, 0, 0, 77, 129, 64)]
    c = Case(spans, 4, 2, 72, "bf16", seed=5, T=spans[-1][1] + 40, layout=layout)
    c.check(**c.places(form, dtype))


@pytest.mark.parametrize("causal", [False, True])
def test_padded_batch_with_other_keys(causal):
    """Sequences of slots with garbage behind them: NaN there reaches nothing, and nothing is written there."""
    spans, keys = [(0, 50), (100, 101), (200, 300), (300, 300), (400, 433)], [(0, 70), (80, 90), (160, 200), (240, 260), (320, 320)]
    c = Case(spans, 2, 1, 64, "f16", seed=2, spans_k=keys, T=500, Tk=400, causal=causal)
    for t, rows in ((c.q, spans), (c.dout, spans), (c.k, keys), (c.v, keys)):
        mine = torch.zeros(t.shape[0], dtype=torch.bool)
        for a, b in rows:
            mine[a:b] = True
        t[~mine.cuda()] = float("nan")
    c.check(**c.places("spans"))


@pytest.mark.parametrize("S", [1, 3, 64, 65, 200])
def test_many_sequences(S):
    """The place of a workgroup is searched for 64 sequences at a time."""
    g = torch.Generator().manual_seed(S)
    spans = cut(*torch.randint(0, 12, (S,), generator=g).tolist())
    if spans[-1][1] == 0:
        spans = cut(*[1] * S)
    c = Case(spans, 1, 1, 16, "bf16", seed=S)
    c.check(**c.places())
    n = spans[-1][1] // 3 * 3
    c = Case(cut(n // 3, n // 3, n // 3), 1, 1, 16, "bf16", seed=S)
    c.check(sequences=3)


def test_thousands_of_sequences():
    spans = cut(*[1 + i % 3 for i in range(5000)])
    c = Case(spans, 1, 1, 8, "bf16", seed=1)
    c.check(**c.places())


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 50)])
@pytest.mark.parametrize("D", [16, 32, 64, 72, 80, 96, 104, 128])
def test_more_tiles_than_cus(D, causal, window):
    """Where workgroups are many, each wave has rows of its own."""
    c = Case(cut(5, 0, 128, 1, 0, 0, 77, 129, 64, 33), 48, 24, D, "bf16" if D % 32 else "f16", seed=D, causal=causal, window=window,
             T=480, layout="rows")
    c.check(**c.places())
    c = Case(cut(160, 160, 160), 96, 96, D, "bf16", seed=D, causal=causal, window=window)
    c.check(sequences=3)


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 50)])
@pytest.mark.parametrize("D", [16, 32, 64, 72, 80, 96, 104, 128])
def test_tiles_enough_for_the_cus(D, causal, window):
    """More tiles yet: none is shared by waves."""
    c = Case(cut(160, 160, 160), 160, 160, D, "bf16" if D % 32 else "f16", seed=D + 1, causal=causal, window=window)
    c.check(sequences=3)
    c = Case(cut(33, 0, 128, 257, 1, 62), 270, 135, D, "bf16", seed=D, causal=causal, window=window, layout="heads")
    c.check(**c.places())


@pytest.mark.parametrize("L,M,H,D,causal,window", [(100, 3501, 512, 104, True, 0), (257, 3700, 256, 128, True, 700),
                                                    (300, 3600, 256, 128, False, 0), (3600, 3600, 40, 112, True, 0)])
def test_long_sequences(L, M, H, D, causal, window):
    """Keys enough for workgroups of eight waves; the definition on the GPU, head by head."""
    c = Case(cut(L), H, 2, D, "bf16", seed=M, spans_k=cut(M), causal=causal, window=window, device="cuda")
    c.check(**c.places())


@pytest.mark.parametrize("spans,spans_k,H,K,D,dt,causal,window", [
    (cut(300), cut(1801), 256, 2, 80, "bf16", False, 0), (cut(700), cut(3700), 200, 4, 96, "f16", True, 1800),
    (cut(513), cut(5000), 256, 1, 72, "bf16", True, 4000), (cut(5400, 0, 1), None, 24, 4, 88, "bf16", False, 0),
    (cut(2050, 1800), None, 80, 8, 128, "f16", False, 1900)])
def test_many_keys(spans, spans_k, H, K, D, dt, causal, window):
    """Queries that see many keys: workgroups of eight waves, for heads of more than 64 elements."""
    c = Case(spans, H, K, D, dt, seed=D, spans_k=spans_k, causal=causal, window=window, device="cuda")
    c.check(**c.places())


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("sigma", [0.0, 0.05, 4.0, 12.0])
def test_flat_and_steep_rows(sigma, dt):
    """Scores from all alike to far apart: the running maximum rises by more and by less than it is followed for."""
    Case(cut(300), 2, 2, 64, dt, seed=3, sigma=sigma).check()


def test_scores_that_rise_and_fall():
    """Keys in the order of their scores, either way, and one far above all others."""
    for order in (1, -1):
        c = Case(cut(400), 1, 1, 32, "bf16", causal=False)
        ramp = torch.linspace(-1, 1, 400, device="cuda")[:, None, None] * order
        c.q.fill_(3.0)
        c.k.copy_(ramp.expand(400, 1, 32) * 2)
        c.k[133] = 5.0
        c.check()


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -20, 0.3])
def test_scales(scale):
    Case(cut(100), 2, 1, 16, "f16", scale=scale).check()


def test_inputs_that_repeat():
    """A stride of 0 gives every head, or every row, the same keys."""
    c = Case(cut(90), 4, 4, 64, "bf16", seed=8)
    c.k = c.k[:, :1].expand(90, 4, 64)
    c.v = c.v[:1].expand(90, 4, 64)
    c.check()


def test_nothing_to_do():
    c = Case([(0, 0)], 2, 2, 64, "bf16", T=0, spans_k=[(0, 4)], Tk=4)
    c.check(**c.places())
    assert (c.dk == 0).all() and (c.dv == 0).all()
    z = Case(cut(4), 2, 2, 64, "bf16")
    none = torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    z.forward(offsets=none)
    z.backward(offsets=none)
    assert (z.out == 3).all() and (z.dq == 3).all() and (z.dk == 3).all()


def test_offsets_out_of_range_touch_nothing_else():
    """Numbers outside the tensor are limited to it; those that fall leave rows unspecified but nothing behind them."""
    for numbers in ([-5, 40, 1000], [0, 1 << 30, 60], [50, 10, 60], [60, 60, 0]):
        c = Case(cut(60), 2, 1, 64, "bf16", seed=4)
        guard = {}
        for x in ("out", "dq", "dk", "dv"):
            n = getattr(c, x)
            buf = torch.full((3, *n.shape), 9.0, dtype=n.dtype, device="cuda")
            guard[x] = buf
            setattr(c, x, buf[1])
        at = torch.tensor(numbers, dtype=torch.int32, device="cuda")
        c.forward(offsets=at)
        c.backward(offsets=at)
        torch.cuda.synchronize()
        for buf in guard.values():
            assert (buf[0] == 9).all() and (buf[2] == 9).all()
    c = Case([(0, 40), (40, 60)], 2, 1, 64, "bf16", seed=4)
    c.check(offsets=torch.tensor([-5, 40, 1000], dtype=torch.int32, device="cuda"))


def test_the_same_bits_again_on_other_streams_and_beside_another_call():
    c = Case(cut(300, 211), 4, 2, 128, "bf16", seed=6)
    other = Case(cut(300, 211), 4, 2, 128, "bf16", seed=7)
    places = c.places()
    c.forward(**places)
    c.backward(**places)
    torch.cuda.synchronize()
    want = [x.clone() for x in (c.out, c.lse, c.dq, c.dk, c.dv)]
    for x in (c.out, c.lse, c.dq, c.dk, c.dv):
        x.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s, case in zip(streams, (c, other)):
        with torch.cuda.stream(s):
            case.forward(**places)
            case.backward(**places)
    torch.cuda.synchronize()
    for x, w in zip((c.out, c.lse, c.dq, c.dk, c.dv), want):
        assert torch.equal(x, w)


def test_captured():
    c = Case(cut(130, 95), 4, 2, 64, "f16", seed=9)
    places = c.places()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        c.forward(**places)
        c.backward(**places)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        c.forward(**places)
        c.backward(**places)
    for i in range(4):
        for x in (c.q, c.k, c.v, c.dout):
            x.copy_(torch.randn(x.shape, device="cuda").to(x.dtype))
        c.forward(**places)
        c.backward(**places)
        torch.cuda.synchronize()
        want = [x.clone() for x in (c.out, c.lse, c.dq, c.dk, c.dv)]
        for x in (c.out, c.lse, c.dq, c.dk, c.dv):
            x.fill_(i)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, w in zip((c.out, c.lse, c.dq, c.dk, c.dv), want):
            assert torch.equal(x, w), i


def test_gradients_against_differences():
    """Central differences of the 64-bit loss around the inputs, in 40 directions: second-order terms of a step h are
    below h^2, so at h = 1e-4 the definition's own gradient agrees to 1e-6; the kernel's is off by its bound, summed
    in the direction."""
    c = Case(cut(40), 2, 1, 16, "f16", seed=11)
    c.check()
    args = (c.spans, c.spans_k, c.causal, c.window, c.scale, c.dt)
    _, bounds = backward(c.q, c.k, c.v, c.out, c.lse, c.dout, *args)
    x = [t.double().cpu() for t in (c.q, c.k, c.v)]
    loss = lambda y: (forward(*y, *args)[0] * c.dout.double().cpu()).sum().item()  # noqa: E731
    g = torch.Generator().manual_seed(1)
    for n in range(40):
        i = n % 3
        d = torch.randn(x[i].shape, generator=g, dtype=torch.float64)
        step = 1e-4 * d
        want = (loss([y + step if j == i else y for j, y in enumerate(x)]) -
                loss([y - step if j == i else y for j, y in enumerate(x)])) / 2e-4
        got = ((c.dq, c.dk, c.dv)[i].double().cpu() * d).sum().item()
        # out was rounded before the backward pass read it: delta is off by u |dout| |out|, ds by p times that
        extra = 2.0 ** -11 * (c.dout.double().cpu().abs() * c.out.double().cpu().abs()).sum(-1).max() * x[1 - min(i, 1)].abs().sum() * c.scale
        assert abs(got - want) <= (bounds[i] * d.abs()).sum().item() + float(extra) * d.abs().max().item() + 1e-5, (n, got, want)


def test_binding_refuses():
    c = Case(cut(10), 4, 2, 16, "bf16")
    f32, out = c.q.float(), c.out
    at = torch.tensor([0, 10], dtype=torch.int32, device="cuda")

    def call(q=c.q, k=c.k, v=c.v, out=out, lse=c.lse, **kw):
        dp.dpa_attention(kw.pop("attention", c.attention), q, k, v, out, lse, **kw)

    for kw in (dict(q=f32), dict(k=c.k.float()), dict(v=c.v[:9]), dict(out=c.out[:, :3]), dict(lse=c.lse[:3]),
               dict(lse=c.lse.double()), dict(q=c.q.cpu()), dict(k=c.k[..., 0]), dict(q=c.q.transpose(1, 2)),
               dict(lse=c.lse.cpu()), dict(offsets=at.cpu()), dict(offsets=torch.zeros(4, dtype=torch.int32, device="cuda")[::2]), dict(offsets=at.float()),
               dict(offsets=at, sequences=2), dict(offsets=at, offsets_k=at.long()),
               dict(offsets=at, offsets_k=torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(sequences=3), dict(k=c.k[:9], v=c.v[:9], offsets=at), dict(out=c.q), dict(k=c.k[:, :0], v=c.v[:, :0]),
               dict(attention=dp.Attention(window=-1)), dict(attention=dp.Attention(scale=-1.0)),
               dict(attention=dp.Attention(scale=0.0)), dict(attention=dp.Attention(scale=float("nan"))),
               dict(out=out[:1].expand(10, 4, 16)), dict(out=out[:, :1].expand(10, 4, 16))):
        with pytest.raises(dp.DpError):
            call(**kw)
    back = [c.q, c.k, c.v, c.out, c.lse, c.dout, c.dq, c.dk, c.dv]
    for i, x, ws in ((6, c.q, c.ws), (7, c.dv, c.ws), (8, c.k, c.ws), (0, c.q, c.ws[:100]), (0, c.q, c.ws[1:])):
        args = list(back)
        args[i] = x
        with pytest.raises(dp.DpError):
            dp.dpa_attention_backward(c.attention, *args, ws)
    assert (c.out == 3).all() and (c.dq == 3).all()


def test_binding_refuses_heads_of_different_sizes():
    c = Case(cut(10), 4, 2, 16, "bf16")
    short, long = (torch.zeros((10, 2, d), dtype=torch.bfloat16, device="cuda") for d in (8, 24))
    for kv in (short, long):
        with pytest.raises(ValueError):
            dp.dpa_attention(c.attention, c.q, kv, kv, c.out, c.lse)
        with pytest.raises(ValueError):
            dp.dpa_attention_backward(c.attention, c.q, kv, kv, c.out, c.lse, c.dout, c.dq, kv.clone(), kv.clone(), c.ws)
    with pytest.raises(ValueError):
        dp.dpa_attention(c.attention, c.q, c.k, short, c.out, c.lse)
    with pytest.raises(ValueError):
        dp.dpa_attention_backward(c.attention, c.q, c.k, c.v, c.out, c.lse, c.dout, c.dq, c.dk, short, c.ws)
    assert (c.out == 3).all() and (c.dq == 3).all() and (c.dk == 3).all()
