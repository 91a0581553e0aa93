"""Scores up to 2^24, where binary32 numbers are one apart: attention on the GPU where each query has keys that score
alike and all others nothing.  Queries and keys are multiples of unit vectors, so every score is exact, the probabilities
are 1 over the number of the visible keys of the query's own direction (e^-score of the others is 0), and out is these
keys' mean.  Bound: p, a multiple of the same power of two in all these keys, is exact or rounded by u, out by u, the sums
add 2 (n + 4) 2^-24 for n keys; lse is a rounding of the score and its sum with log n, 4 2^-24 of it."""
import pytest
import torch

import gradient_reduce_adam_amd as dp
from attention_common import DT, E, U

pytestmark = pytest.mark.gpu

SHAPES = [(40, 200, 2, 1, 16), (257, 257, 4, 2, 64), (200, 300, 300, 300, 40), (150, 700, 700, 700, 80), (64, 64, 900, 900, 128),
          (700, 3700, 256, 4, 128), (600, 3600, 256, 2, 72)]


@pytest.mark.parametrize("dt,power", [("bf16", 5), ("bf16", 9), ("bf16", 12), ("f16", 5), ("f16", 9), ("f16", 12)])
@pytest.mark.parametrize("scale", [0.44, 0.3, 0.29, 0.07])
@pytest.mark.parametrize("L,M,H,K,D", SHAPES)
def test_far_scores(L, M, H, K, D, scale, dt, power):
    A, B = 181 / 128 * 2.0 ** power, 203 / 128 * 2.0 ** power  # A B has 16 bits
    g = torch.Generator(device="cuda").manual_seed(D)
    which_q, which_k = torch.arange(L, device="cuda") * 7 % D, torch.arange(M, device="cuda") % D
    q, k = torch.zeros((L, H, D), device="cuda"), torch.zeros((M, K, D), device="cuda")
    q[torch.arange(L, device="cuda"), :, which_q] = A
    k[torch.arange(M, device="cuda"), :, which_k] = B
    q, k = q.to(DT[dt]), k.to(DT[dt])
    assert scale * A * B < 2 ** 24
    v = torch.randn((M, K, D), generator=g, device="cuda").to(DT[dt])
    out, lse = torch.zeros_like(q), torch.zeros((H, L), device="cuda")
    dp.dpa_attention(dp.Attention(causal=True, scale=scale), q, k, v, out, lse)
    seen = torch.arange(M, device="cuda") <= torch.arange(L, device="cuda")[:, None] + M - L
    own = (which_q[:, None] == which_k) & seen
    count, top = own.sum(1), float(torch.tensor(scale, dtype=torch.float32)) * A * B
    assert (seen.sum(1) >= 1).all()
    weight = torch.where(count[:, None] > 0, own, seen).double()  # without one all score 0
    weight = weight / weight.sum(1, keepdim=True)
    per_key_head = torch.einsum("lm,mkd->lkd", weight, v.double())
    mags = torch.einsum("lm,mkd->lkd", weight, v.double().abs())
    want = per_key_head.repeat_interleave(H // K, 1)
    bound = ((2 * U[dt] + (2 * (M + 4) + 64) * E) * mags + U[dt] * per_key_head.abs() + 2.0 ** -24).repeat_interleave(H // K, 1)
    err = (out.double() - want).abs()
    assert torch.isfinite(out).all() and (err <= bound).all(), (err / bound).max().item()
    want = torch.where(count > 0, top + torch.where(count > 0, count, 1).double().log(), seen.sum(1).double().log())
    assert ((lse.double() - want).abs() <= 6 * E * want.abs() + (M + 8) * E).all()
    dout, dq, dk, dv = torch.randn_like(out), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    ws = torch.empty(dp.dpa_attention_workspace(L, H), dtype=torch.uint8, device="cuda")
    dp.dpa_attention_backward(dp.Attention(causal=True, scale=scale), q, k, v, out, lse, dout, dq, dk, dv, ws)
    assert torch.isfinite(dv).all() and (dv != 0).any()
