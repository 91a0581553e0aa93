"""f16's small numbers in the attention on the GPU: probabilities far below 1, of long rows, keep their bits.

Bounds, u = 2^-11 (half a step of f16) and e = 2^-24.  Flat rows: every p is 1 / M, rounded to f16 with a relative error
of u wherever a power of two brings it into the normal range, the sum over queries and its store add u and 64 e; lse is
off by 2 e of itself, and p with it."""
import math

import pytest
import torch

import gradient_reduce_adam_amd as dp
from attention_common import DT, E

pytestmark = pytest.mark.gpu
U = 2.0 ** -11


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,L,H,K", [(1001, 3, 2, 1), (20011, 40, 2, 2), (100003, 40, 4, 1), (1000003, 33, 1, 1), (70001, 8, 700, 700)])
def test_value_gradients_of_long_flat_rows(M, L, H, K, dt):
    D, u = 8, U if dt == "f16" else 2.0 ** -8
    g = torch.Generator().manual_seed(M)
    q = torch.zeros((L, H, D), dtype=DT[dt], device="cuda")
    k = torch.zeros((M, K, D), dtype=DT[dt], device="cuda")
    # one column for all keys, so that dv is the same in each of them
    v = torch.ones((M, K, D), dtype=DT[dt], device="cuda")
    dout = ((torch.rand((L, H, D), generator=g) + 0.5) * 3e4 / L).to(DT[dt]).cuda()
    out, lse = torch.zeros_like(q), torch.zeros((H, L), device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    ws = torch.empty(dp.dpa_attention_workspace(L, H), dtype=torch.uint8, device="cuda")
    a = dp.Attention()
    dp.dpa_attention(a, q, k, v, out, lse)
    assert torch.equal(out, torch.ones_like(out)) and ((lse.double() - math.log(M)).abs() <= 8 * E * math.log(M)).all()
    dp.dpa_attention_backward(a, q, k, v, out, lse, dout, dq, dk, dv, ws)
    want = dout.double().view(L, K, H // K, D).sum((0, 2)) / M
    err = (dv.double() - want).abs()
    bound = (2 * u + (64 + 4 * math.log(M) + 2 * (L * H // K + 4)) * E) * want + 2.0 ** -25
    assert (err <= bound).all(), (err / bound).max().item()


@pytest.mark.parametrize("H", [1, 260, 700])
@pytest.mark.parametrize("below", [10.0, 14.0, 17.0])
def test_far_keys_behind_a_near_one(below, H):
    """One key above M others whose probabilities are e^-below of its own: together they have a share of the output that
    none of them has bits for, relative to a maximum of 1, in f16's normal range.  Two values, 1 for the first key and 2
    for the others: out = 1 + the others' share; their p is off by u of it.  A sum goes over at most M / 8 partial sums, each
    off by e of a total of 1."""
    M, D = 200001, 8
    k = torch.zeros((M, 1, D), dtype=torch.float16, device="cuda")
    q = torch.zeros((1, H, D), dtype=torch.float16, device="cuda")
    v = torch.full((M, 1, D), 2.0, dtype=torch.float16, device="cuda")
    k[0], q[..., 0], v[0] = 1.0, below, 1.0
    k[0, 0, 1:] = 0
    out, lse = torch.zeros_like(q), torch.zeros((H, 1), device="cuda")
    dp.dpa_attention(dp.Attention(scale=1.0), q, k, v, out, lse)
    share = (M - 1) * math.exp(-below)
    share /= 1 + share
    sums = (M / 8 + 64) * E * (1 + share)
    bound = U * 2 * share + U * (1 + share) + sums
    assert ((out.double() - (1 + share)).abs() <= bound).all(), ((out.double() - 1 - share).abs().max().item(), bound)
    assert ((lse.double() - (below + math.log1p((M - 1) * math.exp(-below)))).abs() <= 64 * E * (below + 1) + sums).all()
