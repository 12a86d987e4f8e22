"""The operators are reached from the package as well as from its functional module."""

import pytest

import lm_head_cross_flce_amd as pkg
from lm_head_cross_flce_amd import functional


@pytest.mark.parametrize("name", [
    "flce_forward", "flce_backward", "flce_linear_forward", "flce_linear_backward", "flce_glu_forward",
    "flce_glu_backward", "flce_grad_norm", "flce_clip_grad_norm", "flce_clip_grads_with_norm", "fused_linear",
    "fused_glu", "GatedFeedForward", "clip_grad_norm_"])
def test_package_exports(name):
    assert getattr(pkg, name) is getattr(functional, name)
