"""What the attention holds of a query: every bf16 value, scaled so that its
row's largest is in [128, 256), as an E4M3 value and an E5M2 value of what is
left.  Values of at least 2^-13 of the largest are exact, and none is off by
more than 2^-21 of it."""

import torch


def test_every_bf16_value():
    v = torch.arange(0x8000, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    v = v[v < 256]                                          # the signs are alike
    half = v.half()
    hi = half.float().to(torch.float8_e4m3fn).float()
    left = (half.float() - hi).half()
    assert torch.equal(left.float(), half.float() - hi)     # the subtraction is exact
    lo = left.float().to(torch.float8_e5m2).float()
    off = (v.double() - hi.double() - lo.double()).abs()
    assert torch.all(off[v >= 2.0 ** -6] == 0)              # 2^-13 of 128, the least that the largest can be
    assert float(off.max()) == 128 * 2.0 ** -21
    assert float(off[(v >= 2.0 ** -7) & (v < 2.0 ** -6)].max()) > 0
