"""The embedding operators on the GPU against plain 64-bit sums.

Tolerances, before any run: a lookup is one binary32 product (2^-24) and one
rounding to the output type (half its epsilon, or half a subnormal step).  A
gradient element is a sum of c products' terms in binary32 in some fixed
order, scaled and added to the accumulator: at most (c - 1) additions, one
product and one addition, each off by 2^-24 of a partial result that is never
more than the sum of magnitudes, so (c + 2) 2^-24 (scale * sum |dy| + |acc|)
(1 + 2^-10) covers every order."""
import numpy as np
import pytest
import torch

import gradient_reduce_adam_amd as dp

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24, "f32": 2.0 ** -149}


def ids_of(kind, T, V, g, dtype=torch.int64):
    if kind == "same":
        x = torch.full((T,), V - 1)
    elif kind == "none":
        x = torch.full((T,), -1)
    elif kind == "sorted":
        x = torch.arange(T) % V
        x = x.sort().values
    elif kind == "reverse":
        x = torch.arange(T - 1, -1, -1) % V
    elif kind == "wild":  # ids far outside the table, and its first and last row
        far = [2 ** 32, -2 ** 40, 2 ** 62] if dtype == torch.int64 else [-2 ** 30, 2 ** 30, 2 ** 31 - 2]
        x = torch.tensor([0, V - 1, V, -1, -2 ** 31, 2 ** 31 - 1] + far)[torch.randint(0, 9, (T,), generator=g)]
    else:  # frequencies that fall with the id, and padding
        u = torch.rand(T, generator=g, dtype=torch.float64)
        x = ((V + 1.0) ** u - 1.0).floor().long().clamp(0, V - 1)
        x = torch.where(torch.rand(T, generator=g) < 0.05, -1, x)
    return x.to(dtype).cuda()


def plain(ids, dy, V, scale):
    """(gradient, sum of magnitudes, token counts) in 64 bits."""
    D = dy.shape[1]
    ok = (ids >= 0) & (ids < V)
    row, d = ids[ok].long(), dy[ok].double()
    g = torch.zeros((V, D), dtype=torch.float64, device="cuda").index_add_(0, row, d)
    m = torch.zeros((V, D), dtype=torch.float64, device="cuda").index_add_(0, row, d.abs())
    c = torch.zeros(V, dtype=torch.float64, device="cuda").index_add_(0, row, torch.ones_like(row, dtype=torch.float64))
    s = float(np.float32(scale))
    return s * g, abs(s) * m, c[:, None]


def check(acc, want, mag, count, before=None):
    base = torch.zeros_like(want) if before is None else before.double()
    tol = (count + 2) * 2.0 ** -24 * (mag + base.abs()) * (1 + 2.0 ** -10) + 2.0 ** -149
    err = (acc.double() - (base + want)).abs()
    assert (err <= tol).all(), f"off by {(err - tol).max().item():.3g} over the bound"


def strided(x, pad):
    """x as a view with `pad` elements between its rows."""
    buf = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=x.dtype, device="cuda")
    buf[:, :x.shape[1]] = x
    return buf[:, :x.shape[1]]


class Setup:
    """A plan of three tensors with the table in the middle, at an element offset of `off`."""

    def __init__(self, V, D, n, off=5, tensors=False, dtype="bf16"):
        self.V, self.D, self.n, self.off = V, D, n, off
        self.numel = (off, V * D, 7)
        self.plan = dp.Plan(self.numel, n, dtype, dtype)
        P = sum(self.numel)
        self.none = torch.zeros(P, dtype=DT[dtype], device="cuda")
        self.acc = [torch.full((P,), 3.25 + r, device="cuda") for r in range(n)]
        for r, a in enumerate(self.acc):
            if tensors:
                self.plan.bind_tensors("acc", [a[0:], a[off:], a[off + V * D:]], r)
            else:
                self.plan.bind("acc", a, r)
            self.plan.bind("grad", self.none, r)

    def table(self, r):
        return self.acc[r][self.off:self.off + self.V * self.D].view(self.V, self.D)

    def outside_untouched(self):
        for r, a in enumerate(self.acc):
            assert (a[:self.off] == 3.25 + r).all() and (a[-7:] == 3.25 + r).all()


def scratch(plan, tensor, D, T):
    return torch.full((max(1, plan.embed_workspace(tensor, D, T)),), 0xAB, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("V,D,T,kind,dt,odt,id_dtype,pad,off", [
    (50, 64, 1, "text", "bf16", "bf16", torch.int64, 0, 0),
    (50, 64, 300, "wild", "bf16", "f32", torch.int32, 0, 8),
    (7, 1, 33, "text", "f16", "f16", torch.int64, 0, 0),
    (300, 37, 129, "wild", "f16", "bf16", torch.int64, 3, 5),
    (100, 768, 257, "text", "bf16", "f16", torch.int32, 8, 8),
    (9, 4104, 17, "text", "f16", "f32", torch.int64, 1, 0),
    (1, 2049, 3, "same", "bf16", "bf16", torch.int64, 0, 3),
    (20, 16, 0, "text", "bf16", "bf16", torch.int64, 0, 0),
])
def test_lookup(V, D, T, kind, dt, odt, id_dtype, pad, off):
    g = torch.Generator().manual_seed(V * 31 + D)
    plan = dp.Plan((off, V * D, 5), 1, dt, dt)
    flat = torch.randn(off + V * D + 5, generator=g).to(DT[dt]).cuda()
    plan.bind("param", flat)
    ids = ids_of(kind, T, V, g, id_dtype)
    out = strided(torch.zeros((T, D), dtype=DT[odt], device="cuda"), pad)
    for scale in (1.0, 0.3):
        plan.embed(1, ids, out, scale=scale)
        ok = (ids >= 0) & (ids < V)
        W = flat[off:off + V * D].view(V, D).double()
        want = W[torch.where(ok, ids, 0).long()] * float(np.float32(scale)) * ok[:, None]
        tol = want.abs() * (torch.finfo(DT[odt]).eps / 2 * 1.001 + 2.0 ** -24) + TINY[odt] / 2
        assert ((out.double() - want).abs() <= tol).all()
        assert (out[~ok] == 0).all()
    if pad and T > 1:
        assert torch.isnan(out.as_strided((T - 1, pad), (D + pad, 1), D)).all()


CASES = [
    # V, D, T, kind, dtype, id type, pad, offset, per-tensor bindings
    (50, 64, 1, "text", "bf16", torch.int64, 0, 8, False),
    (1, 1, 1, "same", "f32", torch.int32, 0, 0, False),
    (3, 5, 2, "text", "f16", torch.int64, 0, 5, False),
    (40, 64, 0, "text", "bf16", torch.int64, 0, 8, False),
    (40, 64, 31, "none", "bf16", torch.int64, 0, 8, False),
    (100, 32, 32, "same", "bf16", torch.int32, 0, 4, False),
    (100, 33, 33, "same", "bf16", torch.int64, 1, 4, True),
    (255, 256, 64, "sorted", "f16", torch.int64, 0, 4, False),
    (256, 257, 65, "reverse", "f16", torch.int32, 0, 1, False),
    (257, 260, 1000, "wild", "f32", torch.int64, 4, 4, False),
    (300, 768, 4095, "text", "bf16", torch.int64, 0, 4, True),
    (65535, 8, 4096, "text", "bf16", torch.int64, 0, 4, False),
    (65536, 12, 4097, "text", "f16", torch.int32, 0, 4, False),
    (70000, 4, 9001, "reverse", "bf16", torch.int64, 0, 4, False),
    (300, 8, 1025, "text", "bf16", torch.int64, 0, 4, False),
    (255, 4, 2049, "same", "f16", torch.int32, 0, 4, False),
    (9000, 12, 8192, "sorted", "bf16", torch.int64, 0, 4, False),
    (9000, 12, 8193, "wild", "f32", torch.int64, 0, 4, False),
    (50257, 8, 16384, "text", "bf16", torch.int32, 0, 4, False),
    (100003, 241, 33, "text", "bf16", torch.int64, 0, 3, False),  # replicas' tables of 289 MB, a ragged end
    (500, 20, 20000, "same", "f32", torch.int64, 0, 4, False),
    (33, 3, 300001, "text", "bf16", torch.int32, 0, 3, False),
]


@pytest.mark.parametrize("V,D,T,kind,dt,id_dtype,pad,off,tensors", CASES)
def test_gradient(V, D, T, kind, dt, id_dtype, pad, off, tensors):
    n = 1 if T > 16384 else 3
    g = torch.Generator().manual_seed(T * 7 + V)
    s = Setup(V, D, n, off, tensors)
    scale = 0.75
    ids = [[ids_of(kind, T, V, g, id_dtype) for _ in range(n)] for _ in range(2)]
    dy = [[strided(torch.randn((T, D), generator=g).to(DT[dt]).cuda(), pad) for _ in range(n)] for _ in range(2)]
    ws = scratch(s.plan, 1, D, T)
    rest = [(0, off), (off + V * D, off + V * D + 7)]

    def micro(k, first):
        s.plan.accumulate_embed(1, ids[k], dy[k], first, ws, scale=scale)

    micro(0, True)
    for r in range(n):
        check(s.table(r), *plain(ids[0][r], dy[0][r], V, scale))
    s.outside_untouched()
    once = [a.clone() for a in s.acc]
    for lo, hi in rest:  # the rest of the micro-step
        s.plan.accumulate_all_range(True, lo, hi)
    micro(1, False)
    for r in range(n):
        before = once[r][off:off + V * D].view(V, D)
        want, mag, count = plain(ids[1][r], dy[1][r], V, scale)
        check(s.table(r), want, mag, count, before)
        idle = (count == 0).expand(V, D)
        assert torch.equal(s.table(r)[idle], before[idle])  # rows without a token keep their bits
    s.plan.close()


def test_same_bits_every_time():
    g = torch.Generator().manual_seed(5)
    V, D, T = 211, 100, 7000
    ids = ids_of("text", T, V, g)
    dy = torch.randn((T, D), generator=g).bfloat16().cuda()
    out = []
    for _ in range(3):
        s = Setup(V, D, 1)
        s.plan.accumulate_embed(1, [ids], [dy], True, scratch(s.plan, 1, D, T))
        out.append(s.table(0).clone())
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])


def test_non_finite_rows_stay_in_their_row():
    V, D, T = 64, 48, 500
    g = torch.Generator().manual_seed(6)
    ids = ids_of("text", T, V, g)
    dy = torch.randn((T, D), generator=g).bfloat16().cuda()
    bad = int((ids == 0).nonzero()[0])
    dy[bad, 3] = float("inf")
    dy[(ids < 0).nonzero()[:, 0]] = float("nan")  # padded positions hold anything
    s = Setup(V, D, 1)
    s.plan.accumulate_embed(1, [ids], [dy], True, scratch(s.plan, 1, D, T))
    finite = torch.isfinite(s.table(0))
    assert not finite[0, 3] and finite.sum() == V * D - 1


def test_two_terms_of_one_tensor():
    """A tied table: two terms in one micro-step add up, in both kinds of micro-step."""
    V, D, T = 90, 36, 200
    g = torch.Generator().manual_seed(7)
    s = Setup(V, D, 2)
    ws = scratch(s.plan, 1, D, T)
    ids = [[ids_of("text", T, V, g) for _ in range(2)] for _ in range(2)]
    dy = [[torch.randn((T, D), generator=g).half().cuda() for _ in range(2)] for _ in range(2)]
    s.plan.accumulate_embed(1, ids[0], dy[0], True, ws, more=True)
    for call in (lambda: s.plan.accumulate_all_range(True, 5, 5 + V * D), lambda: s.plan.accumulate_all(True),
                 lambda: s.plan.accumulate(0, True)):
        with pytest.raises(dp.DpError) as e:
            call()
        assert e.value.status == dp.DP_ERR_STATE
    with pytest.raises(dp.DpError) as e:  # another first flag within the micro-step
        s.plan.accumulate_embed(1, ids[1], dy[1], False, ws)
    assert e.value.status in (dp.DP_ERR_INVALID_ARG, dp.DP_ERR_STATE)
    s.plan.accumulate_embed(1, ids[1], dy[1], True, ws, more=False)
    with pytest.raises(dp.DpError) as e:  # the tensor is covered now
        s.plan.accumulate_embed(1, ids[1], dy[1], True, ws)
    assert e.value.status == dp.DP_ERR_STATE
    for r in range(2):
        a, b = (plain(ids[k][r], dy[k][r], V, 1.0) for k in range(2))
        check(s.table(r), a[0] + b[0], a[1] + b[1], a[2] + b[2])
    s.outside_untouched()


def test_captured_and_replayed():
    V, D, T = 128, 64, 5000
    g = torch.Generator().manual_seed(8)
    s = Setup(V, D, 1, off=8)
    ws = scratch(s.plan, 1, D, T)
    ids, dy = ids_of("text", T, V, g), torch.randn((T, D), generator=g).bfloat16().cuda()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    rest = [(0, 8), (8 + V * D, 8 + V * D + 7)]
    with torch.cuda.stream(stream):
        s.plan.accumulate_embed(1, [ids], [dy], True, ws)
        for lo, hi in rest:
            s.plan.accumulate_all_range(True, lo, hi)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            s.plan.accumulate_embed(1, [ids], [dy], True, ws)
    for k in range(4):
        fresh = ids_of("text", T, V, g)
        ids.copy_(fresh)
        dy.copy_(torch.randn((T, D), generator=g).bfloat16())
        s.acc[0].fill_(-7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(s.table(0), *plain(ids, dy, V, 1.0))
        e = Setup(V, D, 1, off=8)
        e.plan.accumulate_embed(1, [ids], [dy], True, ws)
        torch.cuda.synchronize()
        assert torch.equal(e.table(0), s.table(0))


def test_on_another_stream_with_its_own_workspace():
    V, D, T = 200, 96, 6000
    g = torch.Generator().manual_seed(9)
    runs = []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    data = [(ids_of("text", T, V, g), torch.randn((T, D), generator=g).bfloat16().cuda()) for _ in streams]
    setups = [Setup(V, D, 1) for _ in streams]
    spaces = [scratch(s.plan, 1, D, T) for s in setups]
    torch.cuda.synchronize()
    for st, (ids, dy), s, ws in zip(streams, data, setups, spaces):
        s.plan.accumulate_embed(1, [ids], [dy], True, ws, stream=st)
    torch.cuda.synchronize()
    for (ids, dy), s in zip(data, setups):
        check(s.table(0), *plain(ids, dy, V, 1.0))
