"""Attention, positions and the distillation loss at their limits on the GPU: element offsets beyond 32 bits in every
tensor, against the same rows in small tensors, bit for bit."""
import pytest
import torch

import gradient_reduce_adam_amd as dp

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def far(T, heads, dim, ld):
    """Rows [T, heads, dim] with ld elements between them, in one allocation."""
    buf = torch.zeros((T, ld), dtype=torch.bfloat16, device="cuda")
    return buf[:, :heads * dim].view(T, heads, dim)


def test_attention_rows_beyond_32_bits():
    # 4.3e9 elements a tensor; rows few enough for the same workgroups, and so the same order of sums, as in the small ones
    T, ld, H, K, D = 15000, 290000, 2, 1, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    last = torch.tensor([[5, 70], [T - 300, T]], dtype=torch.int64, device="cuda")
    rows = torch.cat([torch.arange(5, 70), torch.arange(T - 300, T)]).cuda()
    small = torch.tensor([0, 65, 365], dtype=torch.int32, device="cuda")
    a = dp.Attention(causal=True)
    big, few = {}, {}
    for name, n in (("q", H), ("k", K), ("v", K), ("out", H), ("dout", H), ("dq", H), ("dk", K), ("dv", K)):
        big[name] = far(T, n, D, ld)
        few[name] = torch.zeros((365, n, D), dtype=torch.bfloat16, device="cuda")
        if name in ("q", "k", "v", "dout"):
            few[name].copy_(torch.randn(few[name].shape, generator=g, device="cuda"))
            big[name][rows] = few[name]
    for t, places in ((big, dict(offsets=last)), (few, dict(offsets=small))):
        n = t["q"].shape[0]
        t["lse"] = torch.zeros((H, n), device="cuda")
        ws = torch.empty(dp.dpa_attention_workspace(n, H), dtype=torch.uint8, device="cuda")
        dp.dpa_attention(a, t["q"], t["k"], t["v"], t["out"], t["lse"], **places)
        dp.dpa_attention_backward(a, *(t[x] for x in ("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv")), ws, **places)
    for x in ("out", "dq", "dk", "dv"):
        assert torch.equal(big[x][rows], few[x]) and few[x].abs().sum() > 0, x
        assert (big[x][70:T - 300] == 0).all()
    assert torch.equal(big["lse"][:, rows], few["lse"])
    # heads far from each other
    del big
    torch.cuda.empty_cache()
    wide = [torch.zeros((2, 1 << 31), dtype=torch.bfloat16, device="cuda")[:, :365 * D].view(2, 365, D).transpose(0, 1) for _ in range(2)]
    wide[0].copy_(few["q"])
    lse = torch.zeros((2, 365), device="cuda")
    dp.dpa_attention(a, wide[0], few["k"], few["v"], wide[1], lse, offsets=small)
    assert torch.equal(wide[1], few["out"]) and torch.equal(lse, few["lse"])


def test_rotary_rows_beyond_32_bits():
    T, ld = 66000, 65600
    r = dp.Rotary((32,))
    x, y = far(T, 2, 64, ld), far(T, 2, 64, ld)
    g = torch.Generator(device="cuda").manual_seed(2)
    x[-100:] = torch.randn((100, 2, 64), generator=g, device="cuda").bfloat16()
    at = torch.arange(T, device="cuda")
    dp.dpa_rotary(r, at, x, y)
    want = torch.empty((100, 2, 64), dtype=torch.bfloat16, device="cuda")
    dp.dpa_rotary(r, at[-100:], x[-100:], want)
    assert torch.equal(y[-100:], want) and (y[:-100] == 0).all()


def test_logits_beyond_32_bits():
    T, V, top = 87000, 50257, 8  # 4.4e9 logits
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.zeros((T, V), dtype=torch.bfloat16, device="cuda")
    logits[-300:] = torch.randn((300, V), generator=g, device="cuda").bfloat16()
    ids = torch.randint(0, V, (T, top), generator=g, device="cuda")
    teacher = torch.randn((T, top), generator=g, device="cuda")
    d = dp.Distillation(2.0, 0.5, 0.5)
    loss, one = torch.zeros(T, device="cuda"), torch.zeros(300, device="cuda")
    grad = torch.empty((300, V), dtype=torch.bfloat16, device="cuda")
    dp.dpd_distill(d, logits[-300:], teacher[-300:], ids[-300:], one, grad, labels=ids[-300:, 0].contiguous())
    dp.dpd_distill(d, logits, teacher, ids, loss, logits, labels=ids[:, 0].contiguous())
    assert torch.equal(loss[-300:], one) and torch.equal(logits[-300:], grad)
