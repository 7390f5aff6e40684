"""A group's scale, max / 7: the FP32 quotient rounded to 16 bits is the exact quotient's nearest 16-bit number."""
from fractions import Fraction

import pytest
import torch


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_dividing_in_fp32_rounds_once(dtype):
    gen = torch.Generator().manual_seed(1)
    bits = 12 if dtype == torch.float16 else 9
    t = torch.randint(2 ** (bits - 1), 2 ** bits, (400,), generator=gen).double() * 2.0 ** (1 - bits)
    near = (7 * t).float()                                         # quotients next to a tie, and anywhere
    tops = torch.cat((near, torch.nextafter(near, near * 2), torch.nextafter(near, near * 0), torch.rand(400, generator=gen) * 10 + 0.01))
    scale = (tops / 7).to(dtype)
    up, down = torch.nextafter(scale, torch.full_like(scale, 100)), torch.nextafter(scale, torch.zeros_like(scale))
    for top, s, u, d in zip(tops.tolist(), scale.tolist(), up.tolist(), down.tolist()):
        q = Fraction(top) / 7
        off = abs(Fraction(s) - q)
        assert off <= abs(Fraction(u) - q) and off <= abs(Fraction(d) - q)
