"""What the feed-forward autograd functions ask of the library, and what importing the binding needs (CPU)."""

import os
import subprocess
import sys

import pytest
import torch

from lm_head_cross_flce_amd import functional as F


@pytest.fixture
def kept(monkeypatch):
    """The `keep` of each forward call; the outputs are zeros of the right shapes."""
    asked = []

    def linear(x, W, b=None, residual=None, activation="none", keep=False):
        asked.append(keep)
        return x.new_zeros(x.shape[0], W.shape[0]), x.new_zeros(x.shape[0], W.shape[0]) if keep else None

    def glu(x, Wg, Wu, bg=None, bu=None, activation="silu", keep=False):
        asked.append(keep)
        y = x.new_zeros(x.shape[0], Wg.shape[0])
        return (y, y.clone(), y.clone()) if keep else (y, None, None)

    monkeypatch.setattr(F, "flce_linear_forward", linear)
    monkeypatch.setattr(F, "flce_glu_forward", glu)
    return asked


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_nothing_is_kept_without_gradients(kept, mode):
    # an nn.Parameter requires gradients in these modes too, but no backward can follow
    block = F.GatedFeedForward(8, 16, "silu", bias=True)
    x = torch.zeros(3, 8)
    with mode():
        assert not block(x, x).requires_grad
        F.fused_linear(x, block.gate_proj.weight, activation="gelu")
    assert kept == [False] * 3


def test_projections_are_kept_for_a_backward(kept):
    block = F.GatedFeedForward(8, 16, "silu")
    x = torch.zeros(3, 8)
    assert block(x).requires_grad
    F.fused_linear(x, block.gate_proj.weight, activation="gelu")
    F.fused_linear(x, block.gate_proj.weight.detach(), None, torch.zeros(3, 16, requires_grad=True), "gelu")
    with torch.no_grad(), torch.enable_grad():
        block(x)
    # the residual's gradient is dy alone: nothing is kept for it
    assert kept == [True, True, True, False, True, True]
    F.fused_glu(x, block.gate_proj.weight.detach(), block.up_proj.weight.detach())
    assert kept[-1] is False


def test_the_binding_imports_without_a_gpu_build_of_torch():
    # what a build of torch without a GPU lacks, taken away before the import
    code = ("import torch\n"
            "del torch._C._cuda_getCurrentRawStream\n"
            "from lm_head_cross_flce_amd import functional as F\n"
            "for call in (lambda: F.flce_linear_forward(torch.zeros(2, 8), torch.zeros(4, 8)),\n"
            "             lambda: F.flce_grad_norm([torch.zeros(2)])):\n"
            "    try:\n"
            "        call()\n"
            "    except ValueError as e:\n"
            "        assert 'GPU' in str(e)\n"
            "    else:\n"
            "        raise AssertionError\n"
            "print('imported')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr
