"""The weight gradient of a linear layer on the GPU against 64-bit products.

Tolerances, before any run: products of 16-bit values (8 or 11 bits times 4)
are exact in binary32; a sum of T of them in any order and grouping, and the
addition to the accumulator, are off by at most (T + 2) 2^-24 of the sum of the
terms' magnitudes.  A matrix instruction may round each of its partial sums
to less than binary32's nearest, by up to a whole last place, so the bound is
2 (T + 2) 2^-24 (sum |dy| |x| + |acc|)."""
import pytest
import torch

import gradient_reduce_adam_amd as dp

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24


def padded(x, pad, fill):
    buf = torch.full((x.shape[0], x.shape[1] + pad), fill, dtype=x.dtype, device="cuda")
    buf[:, :x.shape[1]] = x
    return buf[:, :x.shape[1]]


class Layer:
    """Operands of one micro-step of n replicas."""

    def __init__(self, T, I, O, n, dt, g, pad=0, spread=4):
        G = -(-I // 32)
        self.dy, self.codes, self.scales, self.x = [], [], [], []
        for _ in range(n):
            dy = torch.randn((T, O), generator=g).to(DT[dt]).cuda()
            codes = torch.randint(0, 256, (T, I), generator=g, dtype=torch.uint8).cuda()
            codes[(codes & 0x7F) == 0x7F] = 0
            scales = torch.randint(127 - spread, 127 + spread - 8, (T, G), generator=g, dtype=torch.uint8).cuda() \
                if spread > 4 else torch.randint(117, 120, (T, G), generator=g, dtype=torch.uint8).cuda()
            e = (scales.double() - 127).repeat_interleave(32, 1)[:, :I]
            self.x.append(codes.view(torch.float8_e4m3fn).double() * torch.exp2(e).round(decimals=30))
            self.dy.append(padded(dy, pad, float("nan")))
            self.codes.append(padded(codes, 2 * pad, 0x7F))
            self.scales.append(padded(scales, pad, 255))

    def want(self, r, transposed):
        d, x = self.dy[r].double(), self.x[r]
        g, m = d.t().contiguous() @ x, d.abs().t().contiguous() @ x.abs()
        return (g.t(), m.t()) if transposed else (g, m)


def check(acc, want, mag, T, before=None):
    base = torch.zeros_like(want) if before is None else before.double()
    tol = 2 * (T + 2) * U * (mag + base.abs()) + 2.0 ** -140
    err = (acc.double() - (base + want)).abs()
    assert torch.isfinite(acc).all() and (err <= tol).all(), \
        f"off by {(err / tol).max().item():.3g} times the bound at {err.argmax().item()}"


class Setup:
    def __init__(self, I, O, n, off=8, tensors=False, dtype="bf16"):
        self.I, self.O, self.n, self.off = I, O, n, off
        self.numel = (off, I * O, 9)
        self.plan = dp.Plan(self.numel, n, dtype, dtype)
        P = sum(self.numel)
        self.none = torch.zeros(P, dtype=DT[dtype], device="cuda")
        self.acc = [torch.full((P,), 1.5 + r, device="cuda") for r in range(n)]
        for r, a in enumerate(self.acc):
            if tensors:
                self.plan.bind_tensors("acc", [a, a[off:], a[off + I * O:]], r)
            else:
                self.plan.bind("acc", a, r)
            self.plan.bind("grad", self.none, r)

    def matrix(self, r, transposed):
        shape = (self.I, self.O) if transposed else (self.O, self.I)
        return self.acc[r][self.off:self.off + self.I * self.O].view(shape)

    def scratch(self, T):
        size = self.plan.linear_workspace(T, self.I, self.O, 1)
        return torch.full((size,), 0xAB, dtype=torch.uint8, device="cuda") if size else None

    def rest(self, first):
        for lo, hi in ((0, self.off), (self.off + self.I * self.O, sum(self.numel))):
            self.plan.accumulate_all_range(first, lo, hi)

    def outside_untouched(self):
        for r, a in enumerate(self.acc):
            assert (a[:self.off] == 1.5 + r).all() and (a[-9:] == 1.5 + r).all()


CASES = [
    # T, I, O, n, pad, off, per-tensor bindings
    (1, 1, 1, 1, 0, 8, False),
    (1, 32, 8, 2, 0, 8, False),
    (2, 5, 3, 2, 0, 3, True),
    (0, 64, 64, 2, 0, 8, False),
    (63, 64, 64, 3, 0, 8, False),
    (64, 256, 256, 1, 0, 8, False),
    (65, 272, 264, 2, 0, 8, False),
    (128, 33, 257, 1, 1, 5, False),
    (129, 512, 40, 3, 8, 8, True),
    (200, 48, 520, 1, 8, 8, False),
    (300, 300, 300, 2, 0, 4, False),
    (1000, 768, 768, 1, 0, 8, False),
    (4097, 256, 520, 1, 0, 8, False),   # split over workgroups
    (1100, 100, 70, 2, 3, 1, False),    # split, no alignment
    (2048, 16, 8, 2, 0, 8, False),
    (640, 2304, 768, 2, 0, 8, False),
]


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,I,O,n,pad,off,tensors", CASES)
def test_gradient(T, I, O, n, pad, off, tensors, dt, transposed):
    g = torch.Generator().manual_seed(T * 13 + I)
    s = Setup(I, O, n, off, tensors)
    ws = s.scratch(T)
    layer = [Layer(T, I, O, n, dt, g, pad) for _ in range(2)]
    before = [None] * n
    for k, first in enumerate((True, False)):
        a = layer[k]
        s.plan.accumulate_linear(1, a.dy, a.codes, a.scales, first, ws, transposed=transposed)
        s.outside_untouched()
        s.rest(first)
        for acc in s.acc:  # the zero gradients of the rest cleared it
            acc[:off], acc[-9:] = 0, 0
        for r in range(n):
            acc = s.matrix(r, transposed)
            check(acc, *a.want(r, transposed), T, before[r])
            before[r] = acc.clone()
        for r, acc in enumerate(s.acc):
            acc[:off], acc[-9:] = 1.5 + r, 1.5 + r


def test_from_packed_activations_and_added_terms():
    """Pack, then the gradient; two terms of one tensor in a micro-step."""
    g = torch.Generator().manual_seed(2)
    T, I, O = 777, 320, 96
    s = Setup(I, O, 1)
    xs, terms = [], []
    for _ in range(2):
        x = (torch.randn((T, I), generator=g) * 3).bfloat16().cuda()
        codes = torch.empty((T, I), dtype=torch.uint8, device="cuda")
        scales = torch.empty((T, I // 32), dtype=torch.uint8, device="cuda")
        dp.dpl_pack_activations(x, codes, scales)
        back = torch.empty_like(x)
        dp.dpl_unpack_activations(codes, scales, back)
        assert ((back.double() - x.double()).abs() <= x.double().abs() * 2.0 ** -4 + 2.0 ** -4).all()
        dy = torch.randn((T, O), generator=g).bfloat16().cuda()
        xs.append(back.double())
        terms.append((dy, codes, scales))
    for k, (dy, codes, scales) in enumerate(terms):
        s.plan.accumulate_linear(1, [dy], [codes], [scales], True, s.scratch(T), more=k == 0)
    want = sum(dy.double().t().contiguous() @ x for (dy, _, _), x in zip(terms, xs))
    mag = sum(dy.double().abs().t().contiguous() @ x.abs() for (dy, _, _), x in zip(terms, xs))
    check(s.matrix(0, False), want, mag, 2 * T)
    with pytest.raises(dp.DpError) as e:
        s.plan.accumulate_linear(1, [terms[0][0]], [terms[0][1]], [terms[0][2]], True, s.scratch(T))
    assert e.value.status == dp.DP_ERR_STATE


def test_non_finite_values_stay_in_their_row_and_column():
    g = torch.Generator().manual_seed(3)
    T, I, O = 130, 300, 280
    for dt in DT:
        a = Layer(T, I, O, 1, dt, g)
        a.codes[0][129, 17] = 0x7F
        a.dy[0][0, 33] = float("inf")
        s = Setup(I, O, 1)
        s.plan.accumulate_linear(1, a.dy, a.codes, a.scales, True, s.scratch(T))
        finite = torch.isfinite(s.matrix(0, False))
        assert not finite[33].any() and not finite[:, 17].any()
        finite[33], finite[:, 17] = True, True
        assert finite.all()


def test_same_bits_and_replays():
    g = torch.Generator().manual_seed(4)
    T, I, O = 5000, 128, 256
    s = Setup(I, O, 1)
    ws = s.scratch(T)
    assert ws is not None  # split over workgroups
    a = Layer(T, I, O, 1, "bf16", g)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        s.plan.accumulate_linear(1, a.dy, a.codes, a.scales, True, ws)
        s.rest(True)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            s.plan.accumulate_linear(1, a.dy, a.codes, a.scales, True, ws)
        s.rest(True)
    for _ in range(3):
        b = Layer(T, I, O, 1, "bf16", g)
        for x, y in zip((a.dy, a.codes, a.scales, a.x), (b.dy, b.codes, b.scales, b.x)):
            x[0].copy_(y[0])
        s.acc[0].fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = s.matrix(0, False).clone()
        check(got, *a.want(0, False), T)
        e = Setup(I, O, 1)
        e.plan.accumulate_linear(1, a.dy, a.codes, a.scales, True, e.scratch(T))
        torch.cuda.synchronize()
        assert torch.equal(e.matrix(0, False), got)
