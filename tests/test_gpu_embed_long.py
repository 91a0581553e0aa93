"""The embedding's gradient from lists that several launches sort: several
replicas with ids of their own, and tables whose ids take one to four digit
passes.  Bounds are those of ``test_gpu_embed.py``."""
import pytest
import torch

from test_gpu_embed import DT, Setup, check, ids_of, plain, scratch, strided

pytestmark = pytest.mark.gpu

CASES = [
    # V, D, T, kinds of the replicas' ids, dtype, id type, pad, offset, per-tensor bindings
    (70000, 4, 20000, ("text", "reverse", "wild"), "bf16", torch.int64, 0, 4, False),   # three passes
    (300, 8, 70001, ("text", "sorted"), "f16", torch.int32, 0, 4, False),               # two passes
    (300, 2, 17000, ("same", "text"), "bf16", torch.int32, 0, 2, False),                # one run through every chunk
    (255, 5, 16385, ("sorted", "text", "none", "reverse"), "f32", torch.int64, 3, 3, True),  # one pass
    (65536, 3, 40000, ("reverse", "text"), "bf16", torch.int32, 1, 1, False),
    ((1 << 24) + 3, 1, 17000, ("text", "reverse"), "f16", torch.int64, 0, 0, False),    # four passes
    ((1 << 24) + 3, 1, 900, ("wild", "text"), "f32", torch.int64, 0, 0, False),         # four passes in one launch
    (1000, 12, 300001, ("text", "text"), "bf16", torch.int64, 0, 4, False),             # spans of several tiles
]


@pytest.mark.parametrize("V,D,T,kinds,dt,id_dtype,pad,off,tensors", CASES)
def test_gradient(V, D, T, kinds, dt, id_dtype, pad, off, tensors):
    n = len(kinds)
    g = torch.Generator().manual_seed(T * 5 + V % 1000)
    s = Setup(V, D, n, off, tensors)
    scale = 0.75
    ids = [[ids_of(kind, T, V, g, id_dtype) for kind in order] for order in (kinds, kinds[::-1])]
    dy = [[strided(torch.randn((T, D), generator=g).to(DT[dt]).cuda(), pad) for _ in range(n)] for _ in range(2)]
    ws = scratch(s.plan, 1, D, T)
    s.plan.accumulate_embed(1, ids[0], dy[0], True, ws, scale=scale)
    for r in range(n):
        check(s.table(r), *plain(ids[0][r], dy[0][r], V, scale))
    s.outside_untouched()
    once = [s.table(r).clone() for r in range(n)]
    for lo, hi in ((0, off), (off + V * D, off + V * D + 7)):
        s.plan.accumulate_all_range(True, lo, hi)
    s.plan.accumulate_embed(1, ids[1], dy[1], False, ws, scale=scale)
    for r in range(n):
        want, mag, count = plain(ids[1][r], dy[1][r], V, scale)
        check(s.table(r), want, mag, count, once[r])
        idle = (count == 0).expand(V, D)
        assert torch.equal(s.table(r)[idle], once[r][idle])  # rows without a token keep their bits
    s.plan.close()


def test_same_bits_from_every_replica():
    """The order of a sum goes by the sizes and the ids alone, whichever replica it belongs to."""
    g = torch.Generator().manual_seed(8)
    V, D, T, n = 70000, 20, 30000, 3
    ids, dy = ids_of("text", T, V, g), torch.randn((T, D), generator=g).bfloat16().cuda()
    s = Setup(V, D, n)
    s.plan.accumulate_embed(1, [ids] * n, [dy] * n, True, scratch(s.plan, 1, D, T))
    assert all(torch.equal(s.table(0), s.table(r)) for r in range(1, n))
    s.plan.close()
