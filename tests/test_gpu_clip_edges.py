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


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("place", ["first", "middle", "last"])
def test_max_norm_of_more_than_the_cache_holds(dt, place):
    # over 160 MB the loads bypass the memory-side cache: the largest element anywhere, of either sign, and a NaN
    n = (200 << 20) // dt.itemsize + 77
    g = rand(n, dt=torch.float32, seed=3).clamp_(-4, 4).to(dt)
    small = rand(1001, seed=4)
    i = {"first": 0, "middle": n // 2, "last": n - 1}[place]
    g[i] = -9.0
    assert float(L.flce_grad_norm([small, g], math.inf)) == 9.0
    norm = L.flce_clip_grad_norm([small, g], 4.5, math.inf)
    assert float(norm) == 9.0
    # 9 * 4.5 / (9 + 1e-6), its product's and its type's rounding
    assert abs(float(g[i]) + 4.5) <= 4.5 * (torch.finfo(dt).eps / 2 + 2.0 ** -22) and float(g.abs().max()) == -float(g[i])
    g[i] = math.nan
    assert math.isnan(float(L.flce_grad_norm([small, g], math.inf)))
    assert math.isnan(float(L.flce_grad_norm([small, g])))
