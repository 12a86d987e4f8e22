"""float32 gelu and its derivative over the whole range, relative to themselves.

Phi(-|z|) is a degree-8 polynomial in t, within 3.8e-7 as evaluated in float32, times exp(-z^2 / 2), whose argument is
kept in two floats: the hardware's exp2 to one step (1.2e-7) and its correction's rounding (6e-8); two more products
(1.2e-7): 6.8e-7 in all, 8e-7 allowed.  For z > 0 Phi is 1 less that, at most 6e-8 more.  Below z = -12.9 the exponential
nears the smallest normal float; the range ends there.
"""

import math

import pytest
import torch

from lm_head_cross_flce_amd import functional as L

pytestmark = pytest.mark.gpu
TOL = 8e-7


def grid():
    return torch.linspace(-12.9, 12.9, 4001, dtype=torch.float64).float()


def phi(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2))


@pytest.mark.parametrize("N", [1, 40, 300])
def test_forward(N):
    z = grid()
    F = z.numel()
    x, W = torch.zeros(N, 8, device="cuda"), torch.zeros(F, 8, device="cuda")
    y, kept = L.flce_linear_forward(x, W, z.cuda(), None, "gelu", keep=True)
    ref = z.double() * phi(z.double())
    assert torch.equal(kept[N - 1].cpu(), z)
    assert bool(((y.double().cpu() - ref).abs() <= TOL * ref.abs()).all())


def test_derivative():
    z = grid()
    F = z.numel()
    x, W = torch.zeros(1, 8, device="cuda"), torch.zeros(F, 8, device="cuda")
    _, kept = L.flce_linear_forward(x, W, z.cuda(), None, "gelu", keep=True)
    _, _, db = L.flce_linear_backward(x, W, torch.ones(1, F, device="cuda"), kept, "gelu", need_db=True)
    d = z.double()
    a, b = phi(d), d * torch.exp(-0.5 * d * d) / math.sqrt(2 * math.pi)
    # the sum's terms, each to TOL, and the sum's rounding
    assert bool(((db.double().cpu() - (a + b)).abs() <= TOL * (a + b.abs()) + 2.0 ** -24 * (a + b).abs()).all())


def test_ends_of_the_range():
    z = torch.tensor([-math.inf, -3e38, -1e20, -100.0, -16.0, -15.0, 15.0, 16.0, 100.0, 1e20, 3e38, math.inf, math.nan])
    F = z.numel()
    x, W = torch.zeros(2, 8, device="cuda"), torch.zeros(F, 8, device="cuda")
    y, kept = L.flce_linear_forward(x, W, z.cuda(), None, "gelu", keep=True)
    _, _, db = L.flce_linear_backward(x[:1], W, torch.ones(1, F, device="cuda"), kept[:1], "gelu", need_db=True)
    y, db = y[0].cpu(), db.cpu()
    assert bool((y[1:6].abs() < 1e-37).all()) and torch.equal(y[6:12], z[6:12]) and bool(torch.isnan(y[12]))
    assert bool((db[1:6].abs() < 1e-37).all()) and torch.equal(db[6:11], torch.ones(5)) and bool(torch.isnan(db[12]))
