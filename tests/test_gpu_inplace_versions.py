"""In-place results count as in-place changes for autograd: a saved tensor that one overwrites is noticed."""

import pytest
import torch

from lm_head_cross_flce_amd import functional as L

pytestmark = pytest.mark.gpu


def test_a_saved_input_used_as_the_output():
    torch.manual_seed(0)
    x = torch.randn(20, 64, device="cuda").requires_grad_(True)
    h = x * 1.0
    W, V = (torch.randn(48, 64, device="cuda").requires_grad_(True) for _ in range(2))
    y = L.fused_glu(h, W, V)
    D = torch.randn(64, 48, device="cuda")
    with torch.no_grad():
        L.flce_linear_forward(y.detach(), D, None, h, out=h)   # the residual stream, in place
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("strided", [False, True])
def test_clipping(strided):
    def grad():
        return torch.randn(30, 80, device="cuda")[:, ::2] if strided else torch.randn(30, 40, device="cuda")

    g, o = grad(), grad()
    before = g._version, o._version
    L.flce_clip_grad_norm([g], 1.0, out=[o])
    assert g._version == before[0] and o._version > before[1]
    L.flce_clip_grad_norm([g], 1.0)
    assert g._version > before[0]
    v = g._version
    L.flce_clip_grads_with_norm([g], 1.0, torch.full((1,), 5.0, device="cuda"))
    assert g._version > v
    v = g._version
    L.flce_grad_norm([g])
    assert g._version == v
    p = torch.nn.Parameter(torch.randn(30, 40, device="cuda"))
    p.grad = grad()
    v = p.grad._version
    L.clip_grad_norm_([p], 0.1)
    assert p.grad._version > v
    with torch.inference_mode():   # tensors without a version
        t = grad()
        L.flce_clip_grad_norm([t], 1.0)
