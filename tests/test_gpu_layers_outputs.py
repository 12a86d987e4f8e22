"""Where the linear layer may write: its own output tensor, also over the residual, and nowhere that it reads."""

import pytest
import torch

from lm_head_cross_flce_amd import _lib
from lm_head_cross_flce_amd import functional as L

pytestmark = pytest.mark.gpu


def randn(*shape, seed, dt=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dt)


@pytest.mark.parametrize("N", [3, 200, 600])
def test_out_over_another_tensor_is_refused(N):
    H = 256
    x, W, b = randn(N, H, seed=1), randn(H, H, seed=2), randn(H, seed=3)
    keep = x.clone()
    with pytest.raises(_lib.FlceError):
        L.flce_linear_forward(x, W, out=x)
    buf = randn(2 * N, H, seed=4)
    with pytest.raises(_lib.FlceError):   # a residual that starts inside out
        L.flce_linear_forward(x, W, None, buf[1:N + 1], out=buf[:N])
    if N <= H:
        with pytest.raises(_lib.FlceError):
            L.flce_linear_forward(x, W, out=W[:N])
    assert torch.equal(x, keep)
    # next to each other in one buffer, and the residual in place: as ever
    ref, _ = L.flce_linear_forward(x, W, b, buf[N:])
    both = torch.cat([x, buf[N:]])
    y, _ = L.flce_linear_forward(both[:N], W, b, both[N:], out=both[N:])
    assert torch.equal(y, ref) and torch.equal(both[:N], x)


def test_equal_weights_are_no_clash():
    x, W = randn(40, 64, seed=1), randn(48, 64, seed=2)
    h, g, u = L.flce_glu_forward(x, W, W, keep=True)
    assert torch.equal(g, u)
    dx, dWg, dWu, _, _ = L.flce_glu_backward(x, W, W, g, u, h)
    assert dWg.data_ptr() != dWu.data_ptr() and dx.shape == x.shape
    x = randn(8, 64, seed=1)   # x its own weights
    y, _ = L.flce_linear_forward(x, x)
    assert torch.equal(y, L.flce_linear_forward(x, x.clone())[0])


def test_both_ways_to_the_current_stream():
    for s in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            assert L._raw_stream(0) == L._current_stream(0) == s.cuda_stream
