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


def test_the_same_strided_memory_twice():
    # gradients whose elements fill no single stretch go through copies, whose addresses differ
    buf = rand(20, 600, seed=2)
    keep = buf.clone()
    for grads in ([buf[:, ::2], buf[:, ::2]], [buf[:, :301], buf[:, 300:]], [buf, buf[:, ::2]]):
        with pytest.raises((ValueError, _lib.FlceError)):
            L.flce_clip_grad_norm(grads, 1.0)
        assert torch.equal(buf, keep)
        with pytest.raises((ValueError, _lib.FlceError)):
            L.flce_clip_grad_norm([g.contiguous() for g in grads], 1.0, out=grads)
        assert torch.equal(buf, keep)
    # side by side in one buffer they are scaled as ever
    n = math.sqrt(float(keep.double().square().sum()))
    norm = L.flce_clip_grad_norm([buf[:, ::2], buf[:, 1::2]], n / 2)
    assert abs(float(norm) - n) <= 2.0 ** -23 * n
    c = (n / 2) / (n + 1e-6)
    assert bool(((buf.double() - keep.double() * c).abs() <= keep.double().abs() * c * 2.0 ** -22).all())
