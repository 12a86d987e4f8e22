"""float16 gradients among the subnormals: operands of the matrix products, not flushed to zero.

dz = dy with no activation, so it is exact; the products are summed in float32 (8 sqrt(K) 2^-24 of the terms' sizes) and
rounded once to float16 (half a step, or half the smallest subnormal).
"""

import math

import pytest
import torch

from lm_head_cross_flce_amd import functional as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tile", ["0", "2", "4", "8"])
@pytest.mark.parametrize("N,H,F", [(3, 64, 48), (70, 264, 100), (600, 512, 640)])
def test_subnormal_gradients(monkeypatch, N, H, F, tile):
    monkeypatch.setenv("FLCE_DEBUG_LAYER_TILE", tile)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (100 * torch.randn(N, H, generator=g, device="cuda")).half()
    W = (100 * torch.randn(F, H, generator=g, device="cuda")).half()
    dy = (2e-6 * torch.randn(N, F, generator=g, device="cuda")).half()   # multiples of 2^-24 of a few units
    assert 0 < float(dy.abs().max()) < 2.0 ** -14
    dx, dW, db = L.flce_linear_backward(x, W, dy, need_db=True)
    d, x64, W64 = dy.double(), x.double(), W.double()
    for got, a, b in ((dx, d, W64), (dW, d.T, x64), (db[:, None], d.T, torch.ones(N, 1, dtype=torch.float64, device="cuda"))):
        ref = a @ b
        tol = 8 * math.sqrt(a.shape[1]) * 2.0 ** -24 * (a.abs() @ b.abs()) + ref.abs() * 2.0 ** -11 + 2.0 ** -25
        assert bool(((got.double() - ref).abs() <= tol).all())
    # the forward: subnormal activations
    small = (x.float() * 2e-8).half()
    y, _ = L.flce_linear_forward(small, W)
    xs = small.double()
    ref = xs @ W64.T
    tol = 8 * math.sqrt(H) * 2.0 ** -24 * (xs.abs() @ W64.abs().T) + ref.abs() * 2.0 ** -11 + 2.0 ** -25
    assert float(xs.abs().max()) < 2.0 ** -14 and bool(((y.double() - ref).abs() <= tol).all())
