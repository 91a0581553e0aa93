"""The norms around a block on the GPU against 64-bit formulas and differences.

Tolerances, before any run.  Outputs are rounded once to their type (half its
epsilon).  What binary32 adds: a row's statistics are sums of D terms in an
unknown order, a relative error of at most (D + 8) 2^-24 in the mean square, half
of it in the factor 1 / sqrt; the mean is off by (D + 2) 2^-24 times the mean
magnitude; a handful of products and sums follow.  So an element of a
normalised row n is off by at most (D + 20) 2^-24 (|n| + m), m the row's mean
magnitude over its deviation (near 1 for these inputs unless the mean is far
from zero), and every later step adds a few 2^-24 of the magnitudes it sums.  The
bound below takes 2 (D + 20) 2^-24 of the sum of the magnitudes that enter an
element, in 64 bits; a column sum over T tokens adds (T + 20) 2^-24 of the sum
of its terms' magnitudes."""
import itertools

import pytest
import torch

import gradient_reduce_adam_amd as dp
from gradient_reduce_adam_amd import BlockNorm

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24
EPS = 1e-5


def strided(x, pad):
    buf = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=x.dtype, device="cuda")
    buf[:, :x.shape[1]] = x
    return buf[:, :x.shape[1]]


def kinds(centered, post, gate, pre):
    names = (["pre_w"] if pre else []) + (["pre_b"] if pre and centered else [])
    names += (["post_w"] if post else []) + (["post_b"] if post and centered else [])
    return names + (["gate"] if gate else [])


class Setup:
    """A plan whose norm tensors lie between two others, at an offset of `off` elements."""

    def __init__(self, D, n, names, dt, pdt, g, centered, alpha, off=8, tensors=False):
        self.D, self.n, self.names, self.off = D, n, names, off
        self.numel = (off,) + (D,) * len(names) + (5,)
        self.plan = dp.Plan(self.numel, n, pdt, pdt)
        P = sum(self.numel)
        self.flat = (torch.randn(P, generator=g) * 0.3 + 1.0).to(DT[pdt]).cuda()
        self.none = torch.zeros(P, dtype=DT[pdt], device="cuda")
        self.acc = [torch.full((P,), 2.5 + r, device="cuda") for r in range(n)]
        starts = [0] + [off + D * i for i in range(len(names) + 1)]
        self.plan.bind("param", self.flat)
        for r, a in enumerate(self.acc):
            if tensors:
                self.plan.bind_tensors("acc", [a[i:] for i in starts], r)
            else:
                self.plan.bind("acc", a, r)
            self.plan.bind("grad", self.none, r)
        self.norms = BlockNorm(centered=centered, eps=EPS, residual_scale=alpha,
                               **{k: i + 1 for i, k in enumerate(names)})
        self.w = {k: self.flat[off + D * i:off + D * (i + 1)].double() for i, k in enumerate(names)}

    def grads(self, r):
        return {k: self.acc[r][self.off + self.D * i:self.off + self.D * (i + 1)] for i, k in enumerate(self.names)}

    def scratch(self, T):
        return torch.full((max(1, self.plan.block_norm_workspace(self.norms, self.D, T)),), 0xAB, dtype=torch.uint8,
                          device="cuda")

    def rest(self, first):
        for lo, hi in ((0, self.off), (self.off + self.D * len(self.names), sum(self.numel))):
            self.plan.accumulate_all_range(first, lo, hi)


def norm(v, w, b, centered):
    """(normalised and scaled, the sum of magnitudes that enters it)."""
    mag = v.abs()
    if centered:
        mag = mag + mag.mean(-1, keepdim=True)
        v = v - v.mean(-1, keepdim=True)
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    out, mag = v * r * w, mag * r * w.abs()
    return (out, mag) if b is None else (out + b, mag + b.abs())


def forward(s, h, y, centered, alpha):
    w = s.w
    h, u = h.double(), y.double()
    mag = u.abs()
    if "post_w" in w:
        u, mag = norm(u, w["post_w"], w.get("post_b"), centered)
    if "gate" in w:
        u, mag = u * w["gate"], mag * w["gate"].abs()
    total, mag = alpha * h + u, abs(alpha) * h.abs() + mag
    if "pre_w" not in w:
        return total, mag, None, None
    x, xm = norm(total, w["pre_w"], w.get("pre_b"), centered)
    # an error in total is carried on as one of the same relative size
    r = torch.rsqrt(((total - (total.mean(-1, keepdim=True) if centered else 0)) ** 2).mean(-1, keepdim=True) + EPS)
    carried = mag * r * w["pre_w"].abs()
    return total, mag, x, 2 * xm + carried + carried.mean(-1, keepdim=True)


def close(got, want, mag, D, dt, extra=0):
    eps = torch.finfo(DT[dt]).eps / 2 if dt else 0.0
    tiny = {"f16": 2.0 ** -25}.get(dt, 2.0 ** -140)
    tol = want.abs() * eps * 1.001 + 2 * (D + 20 + extra) * U * mag + tiny
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all() and (err <= tol).all(), \
        f"off by {(err / tol.clamp(min=1e-300)).max().item():.3g} times the bound"


SHAPES = [(1, 1, 0, 8), (3, 7, 0, 3), (2, 64, 0, 8), (5, 500, 3, 5), (9, 512, 8, 8), (33, 768, 0, 8), (6, 1000, 0, 8),
          (4, 1025, 0, 8), (7, 2048, 0, 8), (5, 2056, 8, 8), (9, 4096, 0, 8), (3, 4099, 0, 1), (2, 8192, 0, 8)]
MODES = [(False, False, False, True, 1.0), (True, False, False, True, 1.0), (False, True, True, True, 0.5),
         (True, True, True, True, -0.7), (False, True, False, False, 1.0), (False, False, True, False, 2.0),
         (True, True, False, True, 0.0)]


@pytest.mark.parametrize("T,D,pad,off", SHAPES)
def test_forward(T, D, pad, off):
    g = torch.Generator().manual_seed(T * 31 + D)
    for i, (centered, post, gate, pre, alpha) in enumerate(MODES):
        dt, pdt = (("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("f32", "f16"))[(i + D) % 4]
        s = Setup(D, 1, kinds(centered, post, gate, pre), dt, pdt, g, centered, alpha, off)
        h, y = (strided((torch.randn((T, D), generator=g) + 0.5).to(DT[dt]).cuda(), pad) for _ in range(2))
        out, x = (strided(torch.zeros((T, D), dtype=DT[dt], device="cuda"), pad) for _ in range(2))
        s.plan.block_norm(s.norms, h, y, out, x if pre else None)
        total, mag, want, xmag = forward(s, h, y, centered, alpha)
        close(out, total, mag, D, dt)
        if pre:
            close(x, want, xmag, D, dt)
        if pad and T > 1:
            assert torch.isnan(out.as_strided((T - 1, pad), (D + pad, 1), D)).all()
        inplace = h.clone() if not pad else strided(h, pad)
        s.plan.block_norm(s.norms, inplace, y, inplace, x if pre else None)  # s in place of h
        assert torch.equal(inplace, out)


def many_rows(T, D, dt, g, n, shift=0.5):
    return [[strided((torch.randn((T, D), generator=g) * f + m).to(DT[dt]).cuda(), 0) for _ in range(n)]
            for f, m in ((1.0, shift), (1.0, shift), (0.1, 0.0), (0.1, 0.0))]


def backward(s, S, Y, dx, ds, centered, alpha):
    """Gradients by the formulas in 64 bits, each with the sum of magnitudes that enters it."""
    w, S, Y = s.w, S.double(), Y.double()
    ds = torch.zeros_like(S) if ds is None else ds.double()
    grads = {}

    def step(v, e, em):
        """(n, magnitude of n, gradient of v from the gradient e of n, its magnitude)."""
        vm = v.abs() + (v.abs().mean(-1, keepdim=True) if centered else 0)
        d = v - v.mean(-1, keepdim=True) if centered else v
        r = torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
        n, nm = d * r, vm * r
        if e is None:
            return n, nm, None, None, r
        c = e - n * (e * n).mean(-1, keepdim=True) - (e.mean(-1, keepdim=True) if centered else 0)
        cm = em + 3 * nm * (em * nm).mean(-1, keepdim=True) + em.mean(-1, keepdim=True)
        return n, nm, r * c, 2 * r * cm, r

    t, tm = ds, ds.abs()
    if "pre_w" in w:
        dx = dx.double()
        n, nm, c, cm, _ = step(S, dx * w["pre_w"], (dx * w["pre_w"]).abs())
        grads["pre_w"] = (dx * n, dx.abs() * nm)
        grads["pre_b"] = (dx, dx.abs())
        t, tm = t + c, tm + cm
    n, nm, u, um = None, None, Y, Y.abs()
    if "post_w" in w:
        n, nm, _, _, _ = step(Y, None, None)
        b = w.get("post_b", torch.zeros_like(w["post_w"]))
        u, um = n * w["post_w"] + b, nm * w["post_w"].abs() + b.abs()
    gate = w.get("gate", torch.ones(s.D, dtype=torch.float64, device="cuda"))
    grads["gate"] = (t * u, tm * um)
    du, dum = t * gate, tm * gate.abs()
    if "post_w" in w:
        grads["post_w"] = (du * n, dum * nm)
        grads["post_b"] = (du, dum)
        _, _, du, dum, _ = step(Y, du * w["post_w"], dum * w["post_w"].abs())
    return alpha * t, abs(alpha) * tm, du, dum, {k: grads[k] for k in s.names}


@pytest.mark.parametrize("T,D,off,n", [(1, 1, 8, 1), (2, 7, 3, 2), (0, 64, 8, 2), (37, 64, 8, 3), (5, 500, 5, 1),
                                       (300, 512, 8, 2), (64, 768, 8, 3), (9, 1000, 8, 2), (700, 1024, 8, 1),
                                       (4, 1025, 8, 1), (30, 2048, 8, 2), (5, 2056, 4, 1), (600, 4096, 8, 1),
                                       (3, 4099, 1, 1), (20, 8192, 8, 1)])
def test_backward(T, D, off, n):
    g = torch.Generator().manual_seed(T * 17 + D)
    for i, (centered, post, gate, pre, alpha) in enumerate(MODES):
        dt, pdt = (("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("f32", "f16"))[(i + T) % 4]
        s = Setup(D, n, kinds(centered, post, gate, pre), dt, pdt, g, centered, alpha, off, tensors=i % 2 == 1)
        ws = s.scratch(T)
        totals = [{k: (torch.zeros(D, dtype=torch.float64, device="cuda"),) * 2 for k in s.names} for _ in range(n)]
        for first in (True, False):
            S, Y, dx, ds = many_rows(T, D, dt, g, n)
            dh, dy = ([torch.full_like(a, 9.0) for a in S] for _ in range(2))
            use_ds = not pre or first
            s.plan.accumulate_block_norm(s.norms, S, Y, dx if pre else None, ds if use_ds else None, dh, dy,
                                         first=first, workspace=ws)
            s.rest(first)
            for r in range(n):
                wh, mh, wy, my, grads = backward(s, S[r], Y[r], dx[r], ds[r] if use_ds else None, centered, alpha)
                close(dh[r], wh, mh, D, dt, 20)
                close(dy[r], wy, my, D, dt, 40)
                for k, acc in s.grads(r).items():
                    a, b = totals[r][k]
                    totals[r][k] = (a + grads[k][0].sum(0), b + grads[k][1].sum(0))
                    close(acc, *totals[r][k], 2 * D + T, None, 60)


def test_gradients_against_differences():
    """The formulas of this file, differentiated numerically in 64 bits."""
    g = torch.Generator().manual_seed(3)
    D, T = 24, 3
    for centered, post, gate, pre, alpha in MODES:
        s = Setup(D, 1, kinds(centered, post, gate, pre), "f32", "bf16", g, centered, alpha)
        h, y, dx, ds = (torch.randn((T, D), generator=g, dtype=torch.float64).cuda() for _ in range(4))

        def loss(h_, y_):
            total, _, x, _ = forward(s, h_, y_, centered, alpha)
            return (total * ds).sum() + (0 if x is None else (x * dx).sum())

        total = forward(s, h, y, centered, alpha)[0]
        dh, _, dy, _, grads = backward(s, total, y, dx, ds, centered, alpha)
        for var, got in ((h, dh), (y, dy)):
            for i, j in itertools.product(range(T), (0, 5, D - 1)):
                old, step = var[i, j].clone(), 1e-6
                var[i, j] = old + step
                up = loss(h, y)
                var[i, j] = old - step
                down = loss(h, y)
                var[i, j] = old
                assert abs((up - down) / (2 * step) - got[i, j]) < 1e-6 * (1 + got[i, j].abs())
        for k in s.names:
            for j in (0, D - 1):
                old, step = s.w[k][j].clone(), 1e-6
                s.w[k][j] = old + step
                up = loss(h, y)
                s.w[k][j] = old - step
                down = loss(h, y)
                s.w[k][j] = old
                want = grads[k][0].sum(0)[j]
                assert abs((up - down) / (2 * step) - want) < 1e-6 * (1 + want.abs())


def test_rows_far_from_zero_and_rows_of_one_value():
    """Deviations, not differences of sums: a mean 1000 times the deviation, and a variance of zero."""
    g = torch.Generator().manual_seed(4)
    D, T = 768, 8
    s = Setup(D, 1, kinds(True, False, False, True), "f32", "bf16", g, True, 1.0)
    h = torch.randn((T, D), generator=g).cuda() + 1000.0
    h[3] = 4.0
    y = torch.zeros_like(h)
    out, x = torch.empty_like(h), torch.empty_like(h)
    s.plan.block_norm(s.norms, h, y, out, x)
    total, mag, want, xmag = forward(s, h, y, True, 1.0)
    close(x, want, xmag, D, "f32")
    # against the naive bound this is the point: the error stays at the mean's rounding, 1000 * 2^-24 * a few
    assert (x[0].double() - want[0]).abs().max() < 64 * 1000 * U
    assert torch.equal(x[3].double(), s.w["pre_b"])


def test_outputs_not_wanted_and_in_place():
    g = torch.Generator().manual_seed(5)
    D, T = 320, 50
    runs = []
    for mode in ("both", "dy only", "dh only", "in place"):
        gg = torch.Generator().manual_seed(6)
        s = Setup(D, 1, kinds(False, True, True, True), "bf16", "bf16", gg, False, 0.5)
        S, Y, dx, ds = many_rows(T, D, "bf16", gg, 1)
        dh, dy = [torch.zeros_like(S[0])], [torch.zeros_like(S[0])]
        if mode == "in place":
            dh, dy = ds, Y
        s.plan.accumulate_block_norm(s.norms, S, Y, dx, ds, None if mode == "dy only" else dh,
                                     None if mode == "dh only" else dy, first=True, workspace=s.scratch(T))
        runs.append((dh[0], dy[0], s.acc[0]))
    assert all(torch.equal(runs[0][2], r[2]) for r in runs)
    assert torch.equal(runs[0][1], runs[1][1]) and torch.equal(runs[0][0], runs[2][0])
    assert torch.equal(runs[0][0], runs[3][0]) and torch.equal(runs[0][1], runs[3][1])


def test_captured_and_replayed():
    g = torch.Generator().manual_seed(7)
    D, T = 512, 700
    s = Setup(D, 1, kinds(True, True, True, True), "bf16", "bf16", g, True, 1.0)
    ws = s.scratch(T)
    data = many_rows(T, D, "bf16", g, 1)
    dh, dy = [torch.zeros_like(data[0][0])], [torch.zeros_like(data[0][0])]
    h, x = torch.zeros_like(dh[0]), torch.zeros_like(dh[0])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())

    def call():
        s.plan.block_norm(s.norms, data[0][0], data[1][0], h, x)
        s.plan.accumulate_block_norm(s.norms, *data, dh, dy, first=True, workspace=ws)

    with torch.cuda.stream(stream):
        call()
        s.rest(True)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call()
        s.rest(True)
    for _ in range(3):
        for a, b in zip(data, many_rows(T, D, "bf16", g, 1)):
            a[0].copy_(b[0])
        for t in (dh[0], dy[0], h, x, s.acc[0]):
            t.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (dh[0], dy[0], h, x, s.acc[0][s.off:-5])]
        call()
        s.rest(True)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (dh[0], dy[0], h, x, s.acc[0][s.off:-5])))


@pytest.mark.parametrize("T,D", [(5000, 512), (4500, 768), (2500, 2048), (1500, 4096), (1300, 4104)])
def test_a_row_does_not_depend_on_the_others(T, D):
    """Workgroups that walk over many rows give each the bits it has in a call of a few rows."""
    g = torch.Generator().manual_seed(8)
    for centered in (False, True):
        s = Setup(D, 1, kinds(centered, True, True, True), "bf16", "bf16", g, centered, 0.5)
        S, Y, dx, ds = many_rows(T, D, "bf16", g, 1)
        ws = s.scratch(T)
        dh, dy, out, x = (torch.zeros_like(S[0]) for _ in range(4))
        s.plan.block_norm(s.norms, S[0], Y[0], out, x)
        s.plan.accumulate_block_norm(s.norms, S, Y, dx, ds, [dh], [dy], first=True, workspace=ws)
        s.rest(True)
        for lo in (0, 300, T - 7):
            part = slice(lo, lo + 7)
            dh2, dy2, out2, x2 = (torch.zeros_like(S[0][part]) for _ in range(4))
            s.plan.block_norm(s.norms, S[0][part], Y[0][part], out2, x2)
            s.plan.accumulate_block_norm(s.norms, *([t[0][part]] for t in (S, Y, dx, ds)), [dh2], [dy2], first=True,
                                         workspace=ws)
            s.rest(True)
            for a, b in ((dh, dh2), (dy, dy2), (out, out2), (x, x2)):
                assert torch.equal(a[part], b)
