"""Every row of a call at the ends of the activations' range, to the types' own precision.

Tolerances: half a step of the type; the activation's relative error (16-bit: 1e-5, from the hardware's exp2 and
reciprocal and the normal distribution's 8.7e-6; float32: 2e-6); and where the sigmoid passes below the smallest normal
float, 2^-126, it may be 0: that is |z| 2^-126 <= 88 * 2^-126 < 1.1e-36 of silu, as |z| <= 88 there and the value falls
from there on.
"""

import math

import pytest
import torch

from lm_head_cross_flce_amd import _lib
from lm_head_cross_flce_amd import functional as L

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def act64(name):
    fn = torch.nn.functional
    return {"none": lambda z: z, "relu": torch.relu, "gelu": fn.gelu, "gelu_tanh": lambda z: fn.gelu(z, approximate="tanh"),
            "silu": fn.silu, "sigmoid": torch.sigmoid}[name]


@pytest.mark.parametrize("tile", ["0", "2"])
@pytest.mark.parametrize("act", tuple(_lib.ACTIVATIONS))
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N", [1, 4, 300, 700])
def test_every_row(monkeypatch, act, dtype, N, tile):
    monkeypatch.setenv("FLCE_DEBUG_LAYER_TILE", tile)
    dt = DT[dtype]
    big = float(torch.finfo(dt).max)
    vals = [0.0, -0.0, 1e-6, -1e-6, 1.0, -1.0, 5.0, -5.0, 20.0, -20.0, 21.0, -21.0, 60.0, -60.0, 90.0, -90.0, 3e4, -3e4,
            big, -big, math.inf, -math.inf, math.nan]
    b = torch.tensor(vals, dtype=dt, device="cuda")
    F = len(vals)
    x, W = torch.zeros(N, 8, dtype=dt, device="cuda"), torch.zeros(F, 8, dtype=dt, device="cuda")
    y, z = L.flce_linear_forward(x, W, b, None, act, keep=True)
    ref = act64(act)(b.double())
    assert torch.equal(torch.isnan(y), torch.isnan(ref).expand_as(y))
    fin = torch.isfinite(ref)
    assert bool((y[:, torch.isinf(ref)] == ref[torch.isinf(ref)]).all())
    tol = ref.abs() * (torch.finfo(dt).eps / 2 + (2e-6 if dt == torch.float32 else 1e-5) * (act != "none")) + TINY[dt] + 1.1e-36
    assert bool(((y.double() - ref).abs() <= tol)[:, fin].all())
    if z is not None:
        assert torch.equal(z.nan_to_num(7.0), b.float().nan_to_num(7.0).expand_as(z))
    h, g, u = L.flce_glu_forward(x, W, W, b, torch.ones_like(b), act, keep=True)
    assert torch.equal(h.nan_to_num(7.0), y.nan_to_num(7.0)) and torch.equal(torch.isnan(h), torch.isnan(y))
    assert torch.equal(u, torch.ones_like(u))
