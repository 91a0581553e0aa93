"""Biases of the block norms, with and without the mean subtracted: every
choice of them next to its weight, forward and backward, against the 64-bit
formulas and under the bounds of ``test_gpu_block_norm.py``.  A bias adds one
product and one sum to an element, which those bounds hold already (they were
derived for norms with biases)."""
import itertools

import pytest
import torch

import gradient_reduce_adam_amd as dp
from gradient_reduce_adam_amd import BlockNorm, driver
from test_gpu_block_norm import DT, Setup, backward, close, forward, many_rows, strided

pytestmark = pytest.mark.gpu

BIASES = [  # the tensors of the norms, in the order of the parameter space
    ("pre_w", "pre_b"),
    ("post_w", "post_b"),
    ("post_w", "post_b", "gate"),
    ("pre_w", "pre_b", "gate"),
    ("pre_w", "post_w", "post_b", "gate"),
    ("pre_w", "pre_b", "post_w"),
    ("pre_w", "pre_b", "post_w", "post_b", "gate"),
    ("pre_w", "post_w", "gate"),
]
KINDS = [("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("f32", "f16")]


@pytest.mark.parametrize("centered", [False, True])
@pytest.mark.parametrize("T,D,pad,off", [(1, 1, 0, 8), (2, 7, 3, 3), (5, 500, 0, 5), (9, 768, 8, 8), (6, 1000, 0, 8),
                                         (7, 2048, 0, 8), (5, 4095, 1, 1), (3, 8192, 0, 8)])
def test_forward(T, D, pad, off, centered):
    g = torch.Generator().manual_seed(T * 37 + D)
    for i, names in enumerate(BIASES):
        dt, pdt = KINDS[(i + D) % 4]
        s = Setup(D, 1, names, dt, pdt, g, centered, 0.5, off)
        h, y = (strided((torch.randn((T, D), generator=g) + 0.5).to(DT[dt]).cuda(), pad) for _ in range(2))
        out, x = (strided(torch.zeros((T, D), dtype=DT[dt], device="cuda"), pad) for _ in range(2))
        s.plan.block_norm(s.norms, h, y, out, x if "pre_w" in names else None)
        total, mag, want, xmag = forward(s, h, y, centered, 0.5)
        close(out, total, mag, D, dt)
        if want is not None:
            close(x, want, xmag, D, dt)


@pytest.mark.parametrize("centered", [False, True])
@pytest.mark.parametrize("T,D,off,n", [(1, 1, 8, 1), (2, 7, 3, 2), (0, 64, 8, 2), (37, 64, 8, 3), (5, 500, 5, 1),
                                       (300, 512, 8, 2), (64, 768, 8, 3), (9, 1000, 8, 2), (30, 2048, 8, 2),
                                       (600, 4096, 8, 1), (3, 4099, 1, 1), (20, 8192, 8, 1)])
def test_backward(T, D, off, n, centered):
    g = torch.Generator().manual_seed(T * 19 + D)
    for i, names in enumerate(BIASES):
        dt, pdt = KINDS[(i + T) % 4]
        s = Setup(D, n, names, dt, pdt, g, centered, -0.7, off, tensors=i % 2 == 1)
        ws = s.scratch(T)
        pre = "pre_w" in names
        totals = [{k: (torch.zeros(D, dtype=torch.float64, device="cuda"),) * 2 for k in s.names} for _ in range(n)]
        for first in (True, False):
            S, Y, dx, ds = many_rows(T, D, dt, g, n)
            dh, dy = ([torch.full_like(a, 9.0) for a in S] for _ in range(2))
            use_ds = not pre or first
            s.plan.accumulate_block_norm(s.norms, S, Y, dx if pre else None, ds if use_ds else None, dh, dy,
                                         first=first, workspace=ws)
            s.rest(first)
            for r in range(n):
                wh, mh, wy, my, grads = backward(s, S[r], Y[r], dx[r], ds[r] if use_ds else None, centered, -0.7)
                close(dh[r], wh, mh, D, dt, 20)
                close(dy[r], wy, my, D, dt, 40)
                for k, acc in s.grads(r).items():
                    a, b = totals[r][k]
                    totals[r][k] = (a + grads[k][0].sum(0), b + grads[k][1].sum(0))
                    close(acc, *totals[r][k], 2 * D + T, None, 60)


def test_gradients_against_differences():
    """The 64-bit formulas with biases, differentiated numerically."""
    g = torch.Generator().manual_seed(13)
    D, T = 24, 3
    for centered, names in itertools.product((False, True), BIASES):
        s = Setup(D, 1, names, "f32", "bf16", g, centered, 0.5)
        h, y, dx, ds = (torch.randn((T, D), generator=g, dtype=torch.float64).cuda() for _ in range(4))

        def loss():
            total, _, x, _ = forward(s, h, y, centered, 0.5)
            return (total * ds).sum() + (0 if x is None else (x * dx).sum())

        total = forward(s, h, y, centered, 0.5)[0]
        _, _, _, _, grads = backward(s, total, y, dx, ds, centered, 0.5)
        for k in s.names:
            for j in (0, D - 1):
                old, step = s.w[k][j].clone(), 1e-6
                s.w[k][j] = old + step
                up = loss()
                s.w[k][j] = old - step
                down = loss()
                s.w[k][j] = old
                want = grads[k][0].sum(0)[j]
                assert abs((up - down) / (2 * step) - want) < 1e-6 * (1 + want.abs())


def test_a_bias_moves_in_a_whole_step():
    """RMS norms whose only upstream gradients are known: after one step every bias has the gradient sum dx, or
    the gate times the sum of what reaches the sum of the rows, and moves by AdamW's first update."""
    D, T = 256, 32
    numel = (D,) * 5
    d = driver.DPStep(numel, 1, 1, "bf16", "bf16", lr=1e-2, weight_decay=0.0)
    g = torch.Generator().manual_seed(2)
    start = (torch.randn(5 * D, generator=g) * 0.1 + 1.0).bfloat16().float().cuda()
    torch.cuda.synchronize()
    d.set_master(lambda ptr: d.master.copy_(start))
    norms = BlockNorm(pre_w=0, pre_b=1, post_w=2, post_b=3, gate=4)
    S, Y, dx, ds = (torch.randn((T, D), generator=g).bfloat16().cuda() for _ in range(4))
    ws = torch.empty(d.plan.block_norm_workspace(norms, D, T), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    d.step_layers(lambda step, k, first, scale: d.plan.accumulate_block_norm(
        norms, [S], [Y], [dx], [ds], None, None, first, ws))
    torch.cuda.synchronize()
    want = dx.double().sum(0)
    got = d.gbar[D:2 * D].double()
    # sums of T bf16 values in binary32, in any order
    assert ((got - want).abs() <= T * 2.0 ** -24 * dx.double().abs().sum(0)).all()
    assert (d.gbar[3 * D:4 * D] != 0).any()
    moved = d.master != start
    assert moved[D:2 * D].float().mean() > 0.9 and moved[3 * D:4 * D].float().mean() > 0.9
    d.close()


def test_one_row_in_place_under_any_stride():
    """A single row has no stride: s in place of h may be given another one."""
    g = torch.Generator().manual_seed(6)
    D = 40
    s = Setup(D, 1, ("pre_w", "post_w"), "bf16", "bf16", g, False, 0.5)
    h, y = (torch.randn((1, D), generator=g).bfloat16().cuda() for _ in range(2))
    out, x, x2 = (torch.zeros_like(h) for _ in range(3))
    s.plan.block_norm(s.norms, h, y, out, x)
    dp._check(dp.lib.dpl_block_norm(s.plan.handle, s.norms.ref(D), 1, dp.DP_BF16, h.data_ptr(), D, y.data_ptr(), D,
                                    h.data_ptr(), D + 8, x2.data_ptr(), D, torch.cuda.current_stream().cuda_stream))
    assert torch.equal(h, out) and torch.equal(x, x2)
