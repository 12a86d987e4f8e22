"""Microscaled tensors of more than 2^31 runs of 8 columns, whose places are counted in 64 bits.

One column is padded to 128, 16 runs, so 2^27 rows of one column pass 2^31 runs with little input.  Such a row has one
element other than zero, and its code and scale depend on that element alone: the rows repeat 1000 values whose codes a
small call gives.
"""

import pytest
import torch

from lm_head_cross_flce_amd import functional as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_places_past_2_to_the_31_runs(fmt):
    R = 2 ** 27 + 4099
    values = torch.randn(1000, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    few = L.flce_mx_quantize(values[:, None], fmt)
    back = L.flce_mx_dequantize(few)
    x = values.repeat(R // 1000 + 1)[:R, None]
    q = L.flce_mx_quantize(x, fmt)
    per, whole = 4_000_000, R - R % 1000     # a whole number of repeats at a time
    for i in range(0, whole, per):
        for got, ref in ((q.codes, few.codes), (q.scales, few.scales)):
            part = got[i:min(i + per, whole)]
            assert torch.equal(part.view(-1, *ref.shape), ref.expand(len(part) // 1000, *ref.shape)), i
    assert torch.equal(q.codes[-(R % 1000):], few.codes[:R % 1000])
    y = L.flce_mx_dequantize(q)
    assert torch.equal(y, back.repeat(R // 1000 + 1, 1)[:R])
