"""The 8-bit activation format on the GPU: every code is pinned.

The format is exact arithmetic but for one rounding to nearest even, so packed
bytes and unpacked values are compared for equality with a definition in
64-bit integers and tables; there is no tolerance."""
import numpy as np
import pytest
import torch

import gradient_reduce_adam_amd as dp

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def e4m3_values():
    """The 127 finite non-negative values of the format, from its definition."""
    v = []
    for code in range(127):
        e, m = code >> 3, code & 7
        v.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v)


VALUES = e4m3_values()


def definition(x, f16):
    """(codes, scale bytes, values) of rows x (float64 array)."""
    T, D = x.shape
    G = -(-D // 32)
    codes, scales = np.zeros((T, D), np.uint8), np.zeros((T, G), np.uint8)
    values = np.zeros((T, D))
    for g in range(G):
        v = x[:, 32 * g:32 * g + 32]
        fin = np.isfinite(v)
        w = np.where(fin, np.clip(v, -61440, 61440) if f16 else v, 0.0)
        top = np.abs(w).max(1)
        e = np.full(T, -117)
        for t in range(T):
            while e[t] < 119 and top[t] > 448.0 * 2.0 ** e[t]:
                e[t] += 1
        q = np.minimum(np.abs(w) / 2.0 ** e[:, None], 448.0)
        hi = np.clip(np.searchsorted(VALUES, q), 1, 126)
        lo = hi - 1
        up = (q - VALUES[lo] > VALUES[hi] - q) | ((q - VALUES[lo] == VALUES[hi] - q) & (hi % 2 == 0))
        c = np.where(up, hi, lo)
        sign = np.signbit(w)
        values[:, 32 * g:32 * g + 32] = np.where(fin, np.where(sign, -1.0, 1.0) * VALUES[c] * 2.0 ** e[:, None], np.nan)
        codes[:, 32 * g:32 * g + 32] = np.where(fin, c | (sign << 7), 0x7F)
        scales[:, g] = e + 127
    return codes, scales, values


def with_pad(x, pad, fill):
    buf = torch.full((x.shape[0], x.shape[1] + pad), fill, dtype=x.dtype, device="cuda")
    buf[:, :x.shape[1]] = x
    return buf, buf[:, :x.shape[1]]


def samples(kind, T, D, dt, g):
    x = torch.randn((T, D), generator=g, dtype=torch.float64)
    if kind == "spread":  # every magnitude that the type has
        lim = {"bf16": 126, "f16": 14, "f32": 126}[dt]
        x = x * 2.0 ** torch.randint(-lim, lim, (T, D), generator=g)
    elif kind == "rows":  # rows of one magnitude each, some of zeros
        lim = {"bf16": 120, "f16": 15, "f32": 120}[dt]
        x = x * 2.0 ** torch.randint(-lim, lim, (T, 1), generator=g)
        x[::5] = 0
    elif kind == "edges":
        pool = torch.tensor([0.0, -0.0, 448, 449, 464, 480, 17 / 16, 19 / 16, 1.75, 1.7578125, 61440, 65504, 2.0 ** -24,
                             3.389e38, -3.389e38, 2.0 ** -126, 2.0 ** -133, float("inf"), -float("inf"), float("nan")],
                            dtype=torch.float64)
        x = pool[torch.randint(0, len(pool), (T, D), generator=g)]
    return x.to(DT[dt]).cuda()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["normal", "spread", "rows", "edges"])
@pytest.mark.parametrize("T,D,pad", [(1, 1, 0), (3, 31, 1), (5, 32, 0), (130, 33, 0), (64, 96, 16), (33, 272, 0),
                                     (7, 1000, 24), (0, 64, 0), (2, 4097, 7)])
def test_pack_and_unpack(dt, kind, T, D, pad):
    g = torch.Generator().manual_seed(T * 100 + D)
    x = samples(kind, T, D, dt, g)
    xb, xv = with_pad(x, pad, 7.0)
    cb, codes = with_pad(torch.zeros((T, D), dtype=torch.uint8, device="cuda"), pad, 0xEE)
    G = -(-D // 32)
    sb, scales = with_pad(torch.zeros((T, G), dtype=torch.uint8, device="cuda"), pad % 3, 0xEE)
    dp.dpl_pack_activations(xv, codes, scales)
    want_c, want_s, want_v = definition(x.double().cpu().numpy().reshape(T, D), dt == "f16")
    assert np.array_equal(scales.cpu().numpy(), want_s)
    got_c = codes.cpu().numpy()
    nan = np.isnan(want_v)
    assert np.array_equal((got_c & 0x7F)[nan], np.full(nan.sum(), 0x7F))
    assert np.array_equal(got_c[~nan], want_c[~nan])
    if pad:  # what lies between the rows is not touched
        assert (cb[:, D:] == 0xEE).all() and (sb[:, G:] == 0xEE).all()
    for odt in DT:
        ob, out = with_pad(torch.zeros((T, D), dtype=DT[odt], device="cuda"), pad, 5.0)
        dp.dpl_unpack_activations(codes, scales, out)
        want = torch.from_numpy(want_v).to(DT[odt])  # exact in the source's own type
        got = out.cpu()
        if odt == dt:
            finite = torch.isfinite(torch.from_numpy(want_v))
            assert torch.equal(want.double()[finite], torch.from_numpy(want_v)[finite])
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got.double(), nan=0.0), torch.nan_to_num(want.double(), nan=0.0))
        if pad:
            assert (ob[:, D:] == 5.0).all()


def test_every_code_unpacks():
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(8, 32)
    v = np.concatenate([VALUES, [np.nan]])
    v = np.concatenate([v, -v]).reshape(8, 32)
    for byte in (10, 118, 127, 200, 246):
        scales = torch.full((8, 1), byte, dtype=torch.uint8, device="cuda")
        out = torch.empty((8, 32), device="cuda")
        dp.dpl_unpack_activations(codes, scales, out)
        want = (v * 2.0 ** (byte - 127)).astype(np.float32)
        assert np.array_equal(out.cpu().numpy(), want, equal_nan=True)
        low = torch.empty((8, 32), dtype=torch.bfloat16, device="cuda")  # a bf16 holds every value
        dp.dpl_unpack_activations(codes, scales, low)
        assert np.array_equal(low.float().cpu().numpy(), want, equal_nan=True)


def test_captured_and_replayed():
    g = torch.Generator().manual_seed(1)
    x = samples("normal", 100, 320, "bf16", g)
    codes = torch.empty((100, 320), dtype=torch.uint8, device="cuda")
    scales = torch.empty((100, 10), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        dp.dpl_pack_activations(x, codes, scales)
        dp.dpl_unpack_activations(codes, scales, out)
    for _ in range(3):
        x.copy_(samples("rows", 100, 320, "bf16", g))
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = definition(x.double().cpu().numpy(), False)[2]
        assert np.array_equal(out.double().cpu().numpy(), want)
