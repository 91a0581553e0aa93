"""The linear weight gradient under every scale of the 8-bit format, and at the
ends of its 16-bit operands' ranges.

One token with dy = 1 makes an element of the gradient the decoded input
itself: code * 2^e rounded once to dy's type (exact in bf16; in f16 to nearest
even, to a subnormal, zero or infinity at its ends).  The sums add zeros only, so the
comparison is for equality."""
import pytest
import torch

import gradient_reduce_adam_amd as dp
from test_gpu_linear import DT, Setup, check, padded

pytestmark = pytest.mark.gpu

SCALES = torch.arange(10, 247, dtype=torch.uint8)  # e from -117 to 119


def operands(lo):
    """Codes lo .. lo + 31 under each of the scales: one row of 32 columns a scale, and the values they stand for."""
    codes = torch.arange(lo, lo + 32, dtype=torch.int64).to(torch.uint8).repeat(len(SCALES))
    value = codes.view(torch.float8_e4m3fn).double() * torch.exp2(SCALES.double() - 127).repeat_interleave(32)
    return codes[None].cuda(), SCALES[None].cuda(), value.cuda()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("transposed", [False, True])
def test_every_code_under_every_scale(dt, transposed):
    O, I = 16, 32 * len(SCALES)
    dy = torch.zeros((1, O), dtype=DT[dt], device="cuda")
    dy[0, 3], dy[0, 9] = 1.0, -2.0
    for lo in range(0, 256, 32):
        codes, scales, value = operands(lo)
        s = Setup(I, O, 1)
        s.plan.accumulate_linear(1, [dy], [codes], [scales], True, s.scratch(1), transposed=transposed)
        g = s.matrix(0, transposed).double()
        g = g.t() if transposed else g
        x = value.float().to(DT[dt])  # binary32 holds every value exactly
        if dt == "bf16":
            assert torch.equal(x.double().nan_to_num(1e300), value.nan_to_num(1e300))
        back = torch.empty((1, I), dtype=DT[dt], device="cuda")
        dp.dpl_unpack_activations(codes, scales, back)
        assert torch.equal(back[0].nan_to_num(nan=7.0, posinf=8.0, neginf=9.0),
                           x.nan_to_num(nan=7.0, posinf=8.0, neginf=9.0)), (dt, lo)
        for row, f in ((3, 1.0), (9, -2.0)):
            want, got = f * x.double(), g[row]
            assert torch.equal(torch.isnan(got), torch.isnan(want)), (dt, lo, row)
            ok = ~torch.isnan(want)
            assert torch.equal(got[ok].float(), want[ok].float()), \
                (dt, lo, row, (got[ok] - want[ok]).abs().nan_to_num(0).max().item())


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_small_output_gradients_keep_their_value(dt):
    """dy down to the smallest numbers of its type, subnormal ones too."""
    tiny = torch.finfo(DT[dt]).tiny * 2.0 ** torch.arange(-12, 12, dtype=torch.float64)
    dy = tiny.to(DT[dt])[None].cuda()
    O, I = dy.shape[1], 32
    codes = torch.full((1, I), 0x38, dtype=torch.uint8, device="cuda")  # 1.0
    e = 100 if dt == "bf16" else 0
    scales = torch.full((1, 1), 127 + e, dtype=torch.uint8, device="cuda")
    s = Setup(I, O, 1)
    s.plan.accumulate_linear(1, [dy], [codes], [scales], True, s.scratch(1))
    want = (dy[0].double() * 2.0 ** e)[:, None].expand(O, I)
    assert torch.equal(s.matrix(0, False).double(), want)


@pytest.mark.parametrize("dt,lo,hi", [("bf16", 87, 168), ("f16", 104, 135)])
def test_mixed_scales_across_tokens(dt, lo, hi):
    """Scales that differ by many powers of two from token to token: the bound goes by the magnitudes in a sum.  In
    f16 a code's value below 2^-14 has fewer bits, which the comparison's own rounding covers."""
    g = torch.Generator().manual_seed(11)
    T, I, O = 300, 200, 130
    dy = padded(torch.randn((T, O), generator=g).to(DT[dt]).cuda(), 3, float("nan"))
    codes = torch.randint(0, 256, (T, I), generator=g, dtype=torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0
    scales = torch.randint(lo, hi, (T, -(-I // 32)), generator=g, dtype=torch.uint8)
    unit = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)[:, :I]
    x = (codes.view(torch.float8_e4m3fn).double() * unit).float().to(DT[dt]).double().cuda()
    assert torch.isfinite(x).all()
    s = Setup(I, O, 1)
    s.plan.accumulate_linear(1, [dy], [padded(codes.cuda(), 5, 0x7F)], [padded(scales.cuda(), 1, 255)], True,
                             s.scratch(T))
    d = dy.double().t().contiguous()
    check(s.matrix(0, False), d @ x, d.abs() @ x.abs(), T)
