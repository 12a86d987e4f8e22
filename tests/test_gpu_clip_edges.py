"""Clipping where its tensors meet: the norm among the gradients, the same memory twice, and large max-norms."""

import math

import pytest
import torch

from lm_head_cross_flce_amd import _lib
from lm_head_cross_flce_amd import functional as L

pytestmark = pytest.mark.gpu


def rand(*shape, dt=torch.float32, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dt)


def test_a_given_norm_inside_a_gradient():
    g = rand(5000, seed=1)
    g[0] = 2.0
    out = torch.empty_like(g)
    L.flce_clip_grads_with_norm([g], 1.0, g[:1], out=[out])   # only read: fine
    # the factor is 1 / (2 + 1e-6): two roundings to float32, of the factor and of the product
    assert bool(((out.double() - g.double() / (2 + 1e-6)).abs() <= g.double().abs() * 2.0 ** -23).all())
    keep = g.clone()
    with pytest.raises(_lib.FlceError):
        L.flce_clip_grads_with_norm([g], 1.0, g[:1])
    with pytest.raises(_lib.FlceError):
        L.flce_clip_grads_with_norm([g], 1.0, out[7:8], out=[out])
    assert torch.equal(g, keep)
