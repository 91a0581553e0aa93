"""Rotary positions on the GPU against complex products in 64 bits.

Bound: the angle is exact to binary64 and reduced there, rounded to binary32 once (2^-24 of at most pi) and its
cosine and sine are off by a few last places of 1: in all 8 2^-24 of the pair's magnitude; two products and a sum
add 3 2^-24, and the result is rounded to the type: half a step."""
import pytest
import torch

import gradient_reduce_adam_amd as dp

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -130, "f16": 2.0 ** -25, "f32": 2.0 ** -140}


def definition(rotary, positions, x, inverse):
    sections, rot = rotary.sections, 2 * sum(rotary.sections)
    x, angle, first = x.double().cpu(), [], 0
    at = positions.cpu().double().view(x.shape[0], len(sections))
    for a, n in enumerate(sections):
        i = torch.arange(n, dtype=torch.float64)
        power = i / n if rotary.own_ladder else (first + i) * 2 / rot
        angle.append(at[:, a, None] * rotary.base ** -power)
        first += n
    turn = torch.polar(torch.ones((), dtype=torch.float64), torch.cat(angle, 1) * (-1 if inverse else 1))[:, None]
    lo, hi = (x[..., 0:rot:2], x[..., 1:rot:2]) if rotary.interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    z = torch.complex(lo.contiguous(), hi.contiguous()) * turn
    y, mag = x.clone(), torch.zeros_like(x)
    at = (slice(0, rot, 2), slice(1, rot, 2)) if rotary.interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    for s, v in zip(at, (z.real, z.imag)):
        y[..., s] = v
        mag[..., s] = torch.maximum(lo.abs(), hi.abs()) * 2 ** 0.5
    return y, mag


def check(rotary, positions, x, y, dt, inverse=False):
    want, mag = definition(rotary, positions, x, inverse)
    tol = 11 * 2.0 ** -24 * mag + U[dt] * (want.abs() + 11 * 2.0 ** -24 * mag) + TINY[dt]
    err = (y.double().cpu() - want).abs()
    assert (err <= tol).all(), (err / tol).max().item()
    rest = 2 * sum(rotary.sections)
    assert torch.equal(y[..., rest:], x[..., rest:])


def rows(T, H, D, dt, seed, layout="own"):
    x = torch.randn((T, H, D), generator=torch.Generator().manual_seed(seed)).to(DT[dt]).cuda()
    if layout == "own":
        return x
    buf = torch.full((T * (H * D + 7) + 1,), 3.0, dtype=x.dtype, device="cuda")
    return buf[1:].view(T, H * D + 7)[:, :H * D].view(T, H, D).copy_(x)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("own_ladder", [False, True])
@pytest.mark.parametrize("sections,D", [((4,), 8), ((32,), 64), ((16, 24, 24), 128), ((3, 0, 5, 2), 23), ((20,), 80),
                                        ((1,), 2), ((5, 4), 19), ((64, 64), 256), ((256,), 512)])
def test_layouts(sections, D, own_ladder, interleaved, dt):
    r = dp.Rotary(sections, 10000.0, interleaved, own_ladder)
    T = 37
    at = torch.randint(-50, 3000, (T, len(sections)), generator=torch.Generator().manual_seed(D)).cuda()
    for layout in ("own", "rows"):
        x, y = rows(T, 3, D, dt, 1, layout), rows(T, 3, D, dt, 2, layout)
        for inverse in (False, True):
            dp.dpa_rotary(r, at, x, y, inverse=inverse)
            check(r, at, x, y, dt, inverse)


@pytest.mark.parametrize("T", [1, 2, 63, 2047, 2048, 5000, 70001])
def test_tokens(T):
    """Workgroups of one token and of several, whole and not."""
    r = dp.Rotary((8,))
    at = torch.arange(T, device="cuda", dtype=torch.int32)
    x = rows(T, 2, 24, "f32", T)
    y = torch.empty_like(x)
    dp.dpa_rotary(r, at, x, y)
    check(r, at, x, y, "f32")


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pairs,D,dt", [(16, 40, "bf16"), (19, 40, "f32")])
def test_outputs_beyond_the_caches(pairs, D, dt, interleaved):
    """More than 64 MiB are written with streaming stores."""
    T, H = 70000, 17
    r = dp.Rotary((pairs,), interleaved=interleaved)
    at = torch.arange(T, device="cuda", dtype=torch.int32)
    x = rows(T, H, D, dt, pairs)
    y = torch.empty_like(x)
    dp.dpa_rotary(r, at, x, y)
    for part in (slice(0, 500), slice(T - 500, T)):
        check(r, at[part], x[part], y[part], dt)
    dp.dpa_rotary(r, at, y, y, inverse=True)
    back = U[dt] * 4 + 64 * 2.0 ** -24
    assert ((y.float() - x.float()).abs().max() <= back * x.float().abs().max() * 2).item()


def test_far_positions_keep_their_phase():
    r = dp.Rotary((16, 16), 500000.0)
    at = torch.tensor([[2 ** 31 - 1, -2 ** 31], [10 ** 6, 2 ** 24 + 1], [2 ** 33 + 3, 12345678]]).cuda()
    x = rows(3, 2, 64, "f32", 1)
    y = torch.empty_like(x)
    dp.dpa_rotary(r, at, x, y)
    # the angle itself is a binary64 product, off by 2^-53 of up to 2^34
    want, mag = definition(r, at, x, False)
    assert ((y.double().cpu() - want).abs() <= 13 * 2.0 ** -24 * mag + 2.0 ** -18 * mag + 2.0 ** -24 * want.abs()).all()


def test_several_tensors_in_place_and_back():
    """Queries and keys of one projection in place, from positions with the axes outside; the inverse undoes it to the
    rounding."""
    T, H, K, D = 77, 6, 2, 48
    r = dp.Rotary((8, 8, 8))
    rows_ = torch.randn((T, (H + 2 * K) * D), generator=torch.Generator().manual_seed(2)).cuda()
    before = rows_.clone()
    q, k = rows_[:, :H * D].view(T, H, D), rows_[:, H * D:(H + K) * D].view(T, K, D)
    at = torch.randint(0, 500, (3, T), generator=torch.Generator().manual_seed(3)).cuda().t()
    dp.dpa_rotary(r, at, (q, k), (q, k))
    check(r, at, before[:, :H * D].view(T, H, D), q, "f32")
    check(r, at, before[:, H * D:(H + K) * D].view(T, K, D), k, "f32")
    assert torch.equal(rows_[:, (H + K) * D:], before[:, (H + K) * D:])
    dp.dpa_rotary(r, at, (q, k), (q, k), inverse=True)
    assert ((rows_ - before).abs().max() <= 32 * 2.0 ** -24 * before.abs().max()).item()


def test_a_row_and_a_head_that_repeat_and_positions_of_one_value():
    x = rows(1, 1, 32, "bf16", 4).expand(40, 5, 32)
    y = torch.empty((40, 5, 32), dtype=torch.bfloat16, device="cuda")
    at = torch.full((1, 1), 9, device="cuda").expand(40, 1)
    r = dp.Rotary((16,))
    dp.dpa_rotary(r, at, x, y)
    check(r, at, x, y, "bf16")


def test_no_pairs():
    x = rows(9, 2, 20, "f16", 5)
    y, at = torch.zeros_like(x), torch.arange(9, device="cuda")
    dp.dpa_rotary(dp.Rotary((0,)), at, x, y)
    assert torch.equal(x, y)
    dp.dpa_rotary(dp.Rotary((0,)), at, x, x)
    assert torch.equal(x, y)


def test_captured():
    r, at = dp.Rotary((16,)), torch.arange(50, device="cuda")
    x = rows(50, 4, 32, "bf16", 1)
    y, stream = torch.empty_like(x), torch.cuda.Stream()
    with torch.cuda.stream(stream):
        dp.dpa_rotary(r, at, x, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        dp.dpa_rotary(r, at, x, y)
    for i in range(3):
        at += i
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(r, at, x, y, "bf16")


def test_binding_refuses():
    x = rows(10, 2, 32, "bf16", 1)
    y, at = torch.full_like(x, 3.0), torch.arange(10, device="cuda")
    r = dp.Rotary((16,))
    for args in ((r, at[:9], x, y), (r, at.float(), x, y), (r, at.cpu(), x, y), (r, at, x, y[:, :1]), (r, at, x, y.float()),
                 (r, at, (x, x), (y,)), (r, at, (x,) * 5, (y,) * 5), (dp.Rotary((4,) * 5), at, x, y), (r, at, x[0], y[0]),
                 (dp.Rotary((8, 8)), at, x, y), (r, at, x.cpu(), y)):
        with pytest.raises(ValueError):
            dp.dpa_rotary(*args)
    for args in ((dp.Rotary((17,)), at, x, y), (dp.Rotary((-1,)), at, x, y), (dp.Rotary((4,), base=0.0), at, x, y),
                 (dp.Rotary((4,), base=float("inf")), at, x, y), (r, at, (x, x), (y, y)), (r, at, (x, y), (y, x)),
                 (r, at, x, y[:1].expand(10, 2, 32))):
        with pytest.raises(dp.DpError):
            dp.dpa_rotary(*args)
    assert (y == 3).all()
    dp.dpa_rotary(r, at[:0], x[:0], y[:0])
