"""The shared expert's weights in 8 bits: rows that vanish or are not finite, as the operators' rows
in 8 bits have them (zero codes, scale 0 or NaN)."""
import math

import pytest
import torch

from weight_only_bit_moe_amd.block import channel_codes


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_that_vanish_or_are_not_finite(dtype):
    g = torch.Generator()
    g.manual_seed(1)
    w = torch.randn(9, 40, generator=g)
    w[0] = 0
    w[1] *= 2.0 ** -130             # 127 / the largest overflows 32 bits
    w[2] *= 2.0 ** -104
    w[3, 7] = math.nan
    w[4, 7] = math.inf
    w[5, 7] = -math.inf
    w[6] *= 2.0 ** -90
    w[7] *= 2.0 ** 120
    w = w.to(dtype)
    q, s = channel_codes(w)
    assert q.dtype == torch.int8 and s.dtype == torch.float32
    assert not q[:6].any()
    assert not s[:3].any() and bool(torch.isnan(s[3:6]).all())
    assert bool((q[6:].abs().amax(1) == 127).all())
    # half a code, and the roundings of the scale, its inverse and the product
    off = (q[6:].double() * s[6:, None].double() - w[6:].double()).abs()
    assert bool((off <= s[6:, None].double() * (0.5 + 127 * 4 * 2.0 ** -24)).all())


def test_codes_are_the_operators():
    """Every step is one FP32 rounding, as in the operators' rows in 8 bits."""
    from tests import _block as R
    g = torch.Generator()
    g.manual_seed(2)
    w = torch.randn(50, 333, generator=g) * torch.exp(3 * torch.randn(50, 1, generator=g))
    q, s = channel_codes(w)
    want, top = R.codes_fp32(w)
    assert torch.equal(q, want) and torch.equal(s, top / 127)


def test_rows_without_elements():
    q, s = channel_codes(torch.empty(0, 8))
    assert q.shape == (0, 8) and s.shape == (0,)
