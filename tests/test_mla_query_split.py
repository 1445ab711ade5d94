"""What the attention holds as the sum of an E4M3 value and an E5M2 value of what
is left, in the arithmetic's definition, over all values.

A query's bf16 values, scaled so that their row's largest is in [128, 256):
those of at least 2^-13 of the largest are exact, and none is off by more than
2^-21 of it.  A probability's fp16 value, up to 2^8.75: within 2^-8 of itself
from 2^-6 on, and never off by more than 2^-14 below that."""

import torch


def parts(half):
    hi = half.float().to(torch.float8_e4m3fn).float()
    left = (half.float() - hi).half()
    assert torch.equal(left.float(), half.float() - hi)     # the subtraction is exact
    return hi.double() + left.float().to(torch.float8_e5m2).double()


def test_every_bf16_value():
    v = torch.arange(0x8000, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    v = v[v < 256]                                          # the signs are alike
    off = (v.double() - parts(v.half())).abs()
    assert torch.all(off[v >= 2.0 ** -6] == 0)              # 2^-13 of 128, the least that the largest can be
    assert float(off.max()) == 128 * 2.0 ** -21
    assert float(off[(v >= 2.0 ** -7) & (v < 2.0 ** -6)].max()) > 0


def test_every_fp16_probability():
    p = torch.arange(0x7C00, dtype=torch.int32).to(torch.int16).view(torch.float16)
    p = p[p <= 2 ** 8.75]
    off = (p.double() - parts(p)).abs()
    assert torch.all(off <= torch.clamp(p.double() * 2.0 ** -8, min=2.0 ** -14))
    assert float(off[p < 2.0 ** -6].max()) == 2.0 ** -14
