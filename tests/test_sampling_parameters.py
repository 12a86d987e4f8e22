"""The sampler's parameters as the library gets them."""

import pytest

from lm_head_cross_flce_amd import _lib


@pytest.mark.parametrize("top_k", [2 ** 63, 2 ** 64 + 5, 10 ** 30])
def test_a_top_k_past_64_bits_is_off(top_k):
    assert _lib.sampling(top_k=top_k).top_k >= 2 ** 31      # longer than any row


@pytest.mark.parametrize("top_k", [-1, -2 ** 63 - 7, -10 ** 30])
def test_a_negative_top_k_is_off(top_k):
    assert _lib.sampling(top_k=top_k).top_k < 0


@pytest.mark.parametrize("top_k", [0, 1, 50, 2 ** 30, 2 ** 40])
def test_others_are_passed_on(top_k):
    assert _lib.sampling(top_k=top_k).top_k == top_k
