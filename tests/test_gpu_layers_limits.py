"""The layer operators at their limits on the GPU: element offsets beyond 32
bits, rows that hold infinities and NaN, and the refusals of the Python
binding."""
import pytest
import torch

import gradient_reduce_adam_amd as dp
from gradient_reduce_adam_amd import BlockNorm

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def test_embedding_table_beyond_32_bits():
    V, D = 1_100_000, 4096  # 4.5e9 elements: 9 GB of parameters, 18 GB of accumulators
    plan = dp.Plan((V * D,), 1)
    param = torch.zeros(V * D, dtype=torch.bfloat16, device="cuda")
    acc = torch.full((V * D,), 7.0, device="cuda")
    plan.bind("param", param)
    plan.bind("acc", acc)
    rows = [0, 1, V // 2, V - 2, V - 1]
    values = torch.arange(1, 6, dtype=torch.bfloat16, device="cuda")
    for i, r in enumerate(rows):
        param.view(V, D)[r] = values[i]
    ids = torch.tensor(rows * 3, device="cuda")
    out = torch.empty((15, D), dtype=torch.bfloat16, device="cuda")
    plan.embed(0, ids, out)
    assert torch.equal(out, values.repeat(3)[:, None].expand(15, D))
    ws = torch.empty(plan.embed_workspace(0, D, 15), dtype=torch.uint8, device="cuda")
    plan.accumulate_embed(0, [ids], [out], True, ws)
    table = acc.view(V, D)
    for i, r in enumerate(rows):
        assert (table[r] == 3 * (i + 1)).all()
    for r in (2, V // 2 - 1, V // 2 + 1, V - 3):
        assert (table[r] == 0).all()
    assert int(torch.count_nonzero(table)) == 5 * D
    plan.accumulate_embed(0, [ids], [out], False, ws)
    assert (table[V - 1] == 30).all() and int(torch.count_nonzero(table)) == 5 * D


def test_rows_beyond_32_bits():
    T, D = 1 << 20, 4104  # 4.3e9 elements a tensor
    g = torch.Generator(device="cuda").manual_seed(1)
    plan = dp.Plan((D, D), 1)
    param = torch.ones(2 * D, dtype=torch.bfloat16, device="cuda")
    plan.bind("param", param)
    acc = torch.empty(2 * D, device="cuda")
    plan.bind("acc", acc)
    norms = BlockNorm(pre_w=0, post_w=1)
    h = torch.zeros((T, D), dtype=torch.bfloat16, device="cuda")
    h[0], h[-1] = 3, torch.randn(D, generator=g, device="cuda").bfloat16()
    s, x = torch.empty_like(h), torch.empty_like(h)
    plan.block_norm(norms, h, h, s, x)
    small = h[[0, -1]].contiguous()
    s2, x2 = torch.empty_like(small), torch.empty_like(small)
    plan.block_norm(norms, small, small, s2, x2)
    assert torch.equal(s[[0, -1]], s2) and torch.equal(x[[0, -1]], x2)
    assert (s[1] == 0).all() and (x[-2] == 0).all()
    # the backward: only the last row has a gradient
    dx = torch.zeros_like(h)
    dx[-1] = 1
    ws = torch.empty(plan.block_norm_workspace(norms, D, T), dtype=torch.uint8, device="cuda")
    dh = torch.empty_like(h)
    plan.accumulate_block_norm(norms, [s], [h], [dx], None, [dh], [x], first=True, workspace=ws)
    got = acc.clone()
    dx2, dh2, dy2 = torch.zeros_like(small), torch.empty_like(small), torch.empty_like(small)
    dx2[1] = 1
    plan.accumulate_block_norm(norms, [s2], [small], [dx2], None, [dh2], [dy2], first=True,
                               workspace=torch.empty(plan.block_norm_workspace(norms, D, 2), dtype=torch.uint8,
                                                     device="cuda"))
    assert torch.equal(dh[-1], dh2[1]) and torch.equal(x[-1], dy2[1]) and torch.equal(got, acc)
    # and packed
    del s, dx, dh
    codes = torch.empty((T, D), dtype=torch.uint8, device="cuda")
    scales = torch.empty((T, 129), dtype=torch.uint8, device="cuda")
    dp.dpl_pack_activations(h, codes, scales)
    x.fill_(9)
    dp.dpl_unpack_activations(codes, scales, x)
    dp.dpl_pack_activations(small, codes[:2], scales[:2])
    dp.dpl_unpack_activations(codes[:2], scales[:2], x2)
    assert torch.equal(x[[0, -1]], x2) and (x[1] == 0).all() and (x[-2] == 0).all()


def test_matrix_beyond_32_bits():
    O, I, T = 70_000, 65_552, 3  # 4.6e9 weights
    plan = dp.Plan((O * I,), 1)
    acc = torch.full((O * I,), 5.0, device="cuda")
    plan.bind("acc", acc)
    dy = torch.zeros((T, O), dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros((T, I), dtype=torch.uint8, device="cuda")
    scales = torch.full((T, -(-I // 32)), 127, dtype=torch.uint8, device="cuda")
    for k, (o, i) in enumerate(((0, 0), (O - 1, I - 1), (O // 2, 1))):
        dy[k, o], codes[k, i] = k + 1, 0x38  # 1.0
    for transposed in (False, True):
        acc.fill_(5.0)
        plan.accumulate_linear(0, [dy], [codes], [scales], True, transposed=transposed)
        m = acc.view(I, O).t() if transposed else acc.view(O, I)
        assert m[0, 0] == 1 and m[O - 1, I - 1] == 2 and m[O // 2, 1] == 3
        assert int(torch.count_nonzero(acc)) == 3


def test_non_finite_rows_stay_in_their_rows():
    g = torch.Generator().manual_seed(2)
    for T, D in ((9, 64), (9, 768), (5, 2048), (4, 4096)):
        plan = dp.Plan((D,) * 5, 1)
        param = torch.ones(5 * D, dtype=torch.bfloat16, device="cuda")
        plan.bind("param", param)
        acc = torch.empty(5 * D, device="cuda")
        plan.bind("acc", acc)
        norms = BlockNorm(pre_w=0, pre_b=1, post_w=2, post_b=3, gate=4, centered=True)
        h, y, dx, ds = (torch.randn((T, D), generator=g).bfloat16().cuda() for _ in range(4))
        h[1, 3], y[2, D - 1], dx[0, 0] = float("inf"), float("nan"), float("inf")
        s, x, dh, dy = (torch.empty_like(h) for _ in range(4))
        plan.block_norm(norms, h, y, s, x)
        fine = torch.isfinite(x).all(1)
        assert not fine[1] and not fine[2] and fine.sum() == T - 2
        s = torch.where(torch.isfinite(s), s, 0)
        y[2, D - 1] = 0
        ws = torch.empty(plan.block_norm_workspace(norms, D, T), dtype=torch.uint8, device="cuda")
        plan.accumulate_block_norm(norms, [s], [y], [dx], [ds], [dh], [dy], first=True, workspace=ws)
        fine = torch.isfinite(dh).all(1) & torch.isfinite(dy).all(1)
        assert not fine[0] and fine[1:].all()
        assert not torch.isfinite(acc[:D]).all()  # the step's check finds it


def test_binding_refusals():
    V, D, T = 30, 32, 8
    plan = dp.Plan((V * D, D, 64 * D), 2)
    param = torch.zeros(V * D + 65 * D, dtype=torch.bfloat16, device="cuda")
    acc = [torch.zeros(V * D + 65 * D, device="cuda") for _ in range(2)]
    plan.bind("param", param)
    for r in range(2):
        plan.bind("acc", acc[r], r)
    ids = torch.zeros(T, dtype=torch.int64, device="cuda")
    out = torch.zeros((T, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    u8 = torch.zeros((T, D), dtype=torch.uint8, device="cuda")
    sc = torch.zeros((T, 1), dtype=torch.uint8, device="cuda")
    dy = torch.zeros((T, 64), dtype=torch.bfloat16, device="cuda")
    n = BlockNorm(pre_w=1)
    calls = [
        lambda: plan.embed(0, ids.cpu(), out),
        lambda: plan.embed(0, ids, out.cpu()),
        lambda: plan.embed(0, ids.float(), out),
        lambda: plan.embed(0, ids[::2], out[:4]),
        lambda: plan.embed(0, ids[:4], out),
        lambda: plan.embed(0, ids, out.t()),
        lambda: plan.embed(0, ids, out.double()),
        lambda: plan.embed(0, ids, out[0]),
        lambda: plan.accumulate_embed(0, [ids], [out], True, ws),
        lambda: plan.accumulate_embed(0, [ids, ids.int()], [out, out], True, ws),
        lambda: plan.accumulate_embed(0, [ids, ids], [out, out.float()], True, ws),
        lambda: plan.accumulate_embed(0, [ids, ids], [out, out[:4]], True, ws),
        lambda: plan.accumulate_embed(0, [ids, ids], [out, torch.zeros((T, 2 * D), dtype=out.dtype, device="cuda")[:, :D]],
                                      True, ws),
        lambda: plan.accumulate_embed(0, [ids, ids], [out, out], True, ws.cpu()),
        lambda: plan.accumulate_embed(0, [ids, ids], [out, out], True, ws[::2]),
        lambda: plan.block_norm(n, out, out[:4], out, out),
        lambda: plan.block_norm(n, out, out.half(), out, out),
        lambda: plan.accumulate_block_norm(n, None, None, None, None, None, None, True, ws),
        lambda: plan.accumulate_block_norm(n, [out], None, [out], None, None, None, True, ws),
        lambda: dp.dpl_pack_activations(out, u8, sc.t()),
        lambda: dp.dpl_pack_activations(out, u8.view(torch.int8), sc),
        lambda: dp.dpl_pack_activations(out, u8[:4], sc),
        lambda: dp.dpl_unpack_activations(u8, torch.zeros((T, 2), dtype=torch.uint8, device="cuda"), out),
        lambda: plan.accumulate_linear(2, [dy, dy], [u8, u8], [sc, sc[:4]], True),
        lambda: plan.accumulate_linear(2, [dy], [u8], [sc], True),
    ]
    for call in calls:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: plan.accumulate_embed(0, [ids, ids], [out, out], True, ws[1:]),
                 lambda: plan.accumulate_embed(0, [ids, ids], [out, out], True, ws[:256]),
                 lambda: plan.accumulate_linear(2, [dy.float()] * 2, [u8, u8], [sc, sc], True),
                 lambda: plan.linear_workspace(8, 7, 9)):
        with pytest.raises(dp.DpError) as e:
            call()
        assert e.value.status == dp.DP_ERR_INVALID_ARG
    # none of them counted as part of a micro-step
    for r in range(2):
        plan.bind("grad", param, r)
    plan.accumulate_all(True)
