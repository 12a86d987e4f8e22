"""Sampling where most of a long row's tokens have weights that are small beside the largest.

Rows of more than 2^18 tokens that are walked whole hold weights as whole numbers of 2^-s, s = 62 - e for a bound in
[2^(e - 1), 2^e) on the sum, 32 times the weights of the largest of each 32 tokens: here 32 and a little, so e = 6.  Where
all tokens but one have the same weight, their roundings of 2^-57 add up, to V 2^-57 at most: the tests say how many tokens
that is.
"""

import math

import pytest
import torch

from lm_head_cross_flce_amd import functional as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [2 ** 24, 2 ** 26])
@pytest.mark.parametrize("how", ["top_p", "top_k"])
def test_a_long_tail_of_small_weights(V, how):
    # one token 27.5 above all others, which have 2^-15.7 (V = 2^24) of the sum together
    z = torch.zeros(8, V, device="cuda")
    z[:, 0] = 27.5
    w = math.exp(-27.5)
    u = torch.tensor([0.0, 0.5, 1 - 2.0 ** -14, 1 - 2.0 ** -16, 1 - 2.0 ** -17, 1 - 2.0 ** -18, 1 - 2.0 ** -20, 1 - 2.0 ** -24],
                     device="cuda")
    if how == "top_p":
        p = 1 - 2.0 ** -24
        tail = math.ceil((p * (1 + (V - 1) * w) - 1) / w)
        got = L.flce_sample(z, u, top_p=p).tolist()
    else:
        tail = V // 3
        got = L.flce_sample(z, u, top_k=tail + 1).tolist()
    # each weight is off by 2^-57 at most: by so many tokens after V of them, in the cut and in the draw
    slack = 2 * V * 2.0 ** -57 / w + 2
    for t, v in zip(got, u.tolist()):
        spot = v * (1 + tail * w)
        want = 0 if spot < 1 else 1 + int((spot - 1) / w)
        assert abs(t - want) <= slack, (v, t, want)
