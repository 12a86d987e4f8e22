"""Refusals of the feed-forward and gradient-clipping entry points, without a GPU.

Every call below carries one invalid argument that validation must catch
before anything is enqueued; the placeholder addresses are never dereferenced.
"""

import ctypes
import math
import os

import pytest
import torch

from lm_head_cross_flce_amd import _lib
from lm_head_cross_flce_amd import functional as F

P = 0x100000      # 256-byte aligned placeholders
P2 = 0x200000
BIG = 1 << 40

INVALID, UNSUPPORTED, TOO_SMALL = (_lib.FLCE_ERR_INVALID_ARGUMENT, _lib.FLCE_ERR_UNSUPPORTED,
                                   _lib.FLCE_ERR_WORKSPACE_TOO_SMALL)


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from lm_head_cross_flce_amd import build
        build.build()
    return _lib.load()


def refused(fn, status, **over):
    with pytest.raises(_lib.FlceError) as e:
        fn(**over)
    assert e.value.status == status, (over, e.value.status)


def linear_fwd(**o):
    a = dict(x=P, W=P, b=None, residual=None, N=100, H=4096, F=256, dtype=1, activation=4, y=P2, z=P2, workspace=P2,
             workspace_bytes=BIG, stream=None)
    a.update(o)
    _lib.flce_linear_forward(**a)


def linear_bwd(**o):
    a = dict(x=P, W=P, z=P, dy=P, N=100, H=4096, F=256, dtype=1, activation=4, dx=P2, dW=P2, db=P2, workspace=P2,
             workspace_bytes=BIG, stream=None)
    a.update(o)
    _lib.flce_linear_backward(**a)


def glu_fwd(**o):
    a = dict(x=P, Wg=P, Wu=P, bg=None, bu=None, N=100, H=4096, F=256, dtype=1, activation=4, h=P2, g=P2, u=P2,
             workspace=P2, workspace_bytes=BIG, stream=None)
    a.update(o)
    _lib.flce_glu_forward(**a)


def glu_bwd(**o):
    a = dict(x=P, Wg=P, Wu=P, g=P, u=P, dh=P, N=100, H=4096, F=256, dtype=1, activation=4, dx=P2, dWg=P2, dWu=P2,
             dbg=P2, dbu=P2, workspace=P2, workspace_bytes=BIG, stream=None)
    a.update(o)
    _lib.flce_glu_backward(**a)


@pytest.mark.parametrize("fn", [linear_fwd, linear_bwd, glu_fwd, glu_bwd])
def test_layer_sizes_and_enums(fn):
    refused(fn, INVALID, N=-1)
    refused(fn, INVALID, H=0)
    refused(fn, INVALID, F=0)
    refused(fn, UNSUPPORTED, H=1 << 21)
    refused(fn, UNSUPPORTED, F=1 << 21)
    refused(fn, UNSUPPORTED, N=1 << 31)
    refused(fn, UNSUPPORTED, N=1 << 30, F=1 << 19)   # the plane of output tiles
    refused(fn, UNSUPPORTED, dtype=3)
    refused(fn, INVALID, activation=6)
    refused(fn, INVALID, activation=-1)


@pytest.mark.parametrize("fn,names", [
    (linear_fwd, ("x", "W", "y")), (linear_bwd, ("x", "W", "z", "dy")), (glu_fwd, ("x", "Wg", "Wu", "h")),
    (glu_bwd, ("x", "Wg", "Wu", "g", "u", "dh"))])
def test_layer_tensors(fn, names):
    for n in names:
        refused(fn, INVALID, **{n: None})
        refused(fn, INVALID, **{n: P + 8})
    opt = {linear_fwd: ("residual", "z"), linear_bwd: ("dx", "dW"), glu_fwd: ("g", "u"), glu_bwd: ("dx", "dWg", "dWu")}
    for n in opt[fn]:
        refused(fn, INVALID, **{n: P2 + 8})
    bias = {linear_fwd: ("b",), linear_bwd: ("db",), glu_fwd: ("bg", "bu"), glu_bwd: ("dbg", "dbu")}
    for n in bias[fn]:
        refused(fn, INVALID, **{n: P2 + 1})


def test_glu_keeps_both_projections_or_none():
    refused(glu_fwd, INVALID, g=None)
    refused(glu_fwd, INVALID, u=None)


@pytest.mark.parametrize("fn", [linear_fwd, linear_bwd, glu_fwd, glu_bwd])
def test_layer_workspace(fn):
    # 100 x 256 outputs over H = 4096: one or two tiles, so both directions need a workspace
    sizes = (_lib.flce_glu_workspace_size(100, 4096, 256, 1) if fn in (glu_fwd, glu_bwd)
             else _lib.flce_linear_workspace_size(100, 4096, 256, 1, 4))
    need = sizes[fn in (linear_bwd, glu_bwd)]
    assert need > 0
    refused(fn, TOO_SMALL, workspace_bytes=need - 1)
    refused(fn, INVALID, workspace=None)
    refused(fn, INVALID, workspace=P2 + 8)


def test_layer_workspace_arithmetic():
    # many tiles: no partial sums; the backward holds dz and the bias sums
    f, b = _lib.flce_linear_workspace_size(8192, 4096, 12288, 1, 4)
    assert f == 0 and 8192 * 12288 * 2 <= b <= 8192 * 12288 * 2 + 128 * 12288 * 4 + 512
    f, b = _lib.flce_linear_workspace_size(8192, 4096, 12288, 1, 0)   # dz is dy
    assert f == 0 and b <= 128 * 12288 * 4 + 512
    f, b = _lib.flce_glu_workspace_size(8192, 4096, 12288, 1)
    assert f == 0 and 2 * 8192 * 12288 * 2 <= b <= 2 * 8192 * 12288 * 2 + 2 * 128 * 12288 * 4 + 512
    # rows of no whole 16-byte pieces: padded copies of x and the weights in both
    a, b = _lib.flce_glu_workspace_size(300, 61, 40, 1), _lib.flce_glu_workspace_size(300, 64, 40, 1)
    assert all(380 * 64 * 2 <= p - q <= 380 * 64 * 2 + 512 for p, q in zip(a, b))
    # no rows: nothing
    assert _lib.flce_linear_workspace_size(0, 64, 64, 1, 4)[0] == 0
    for bad in ((-1, 64, 64), (4, 0, 64), (4, 64, 0)):
        with pytest.raises(_lib.FlceError):
            _lib.flce_linear_workspace_size(*bad, 1, 0)
        with pytest.raises(_lib.FlceError):
            _lib.flce_glu_workspace_size(*bad, 1)


def clip(grads=(P, P2), outs=None, numels=(16, 16), dtypes=(0, 1), count=2, max_norm=1.0, norm_type=2.0, norm=P,
         workspace=P, workspace_bytes=BIG, arrays=True):
    _lib.flce_clip_grad_norm(_lib.pointer_array(grads) if arrays else None,
                             None if outs is None else _lib.pointer_array(outs), _lib.size_array(numels),
                             _lib.dtype_array(dtypes), count, max_norm, norm_type, norm, workspace, workspace_bytes, None)


def test_clip_arguments():
    refused(clip, INVALID, count=-1)
    refused(clip, INVALID, count=(1 << 20) + 1)
    refused(clip, INVALID, arrays=False)
    refused(clip, INVALID, numels=(16, -1))
    refused(clip, INVALID, grads=(P, 0))
    refused(clip, INVALID, grads=(P, P2 + 1))
    refused(clip, INVALID, grads=(P + 2, P2))        # float32 at a 2-byte boundary
    refused(clip, UNSUPPORTED, dtypes=(0, 7))
    refused(clip, UNSUPPORTED, norm_type=1.0)
    refused(clip, UNSUPPORTED, norm_type=-math.inf)
    refused(clip, UNSUPPORTED, norm_type=math.nan)
    refused(clip, INVALID, max_norm=-1.0)
    refused(clip, INVALID, max_norm=math.nan)
    refused(clip, INVALID, norm=None)
    refused(clip, INVALID, norm=P + 2)
    refused(clip, INVALID, workspace=None)
    refused(clip, TOO_SMALL, workspace_bytes=_lib.flce_grad_norm_workspace_size(2) - 1)


def test_clip_refuses_shared_memory():
    refused(clip, INVALID, grads=(P, P))                              # the same tensor twice
    refused(clip, INVALID, grads=(P, P + 60))                         # the last float32 of the first
    refused(clip, INVALID, outs=(P2 + 32, P2 + 64), grads=(P, P2))    # one's out over the other's gradient
    refused(clip, INVALID, outs=(P + 4, P2))                          # an out over its own gradient, shifted
    refused(clip, INVALID, outs=(P + 4096, P + 4096))                 # two outs in one place
    refused(clip, INVALID, outs=(0, P2))
    refused(clip, INVALID, outs=(P + 2, P2))
    # an output inside a long gradient that another, shorter one separates from it in address order
    refused(clip, INVALID, grads=(P, P + 4096), outs=(P2, P + 8192), numels=(1 << 14, 16))


def test_clip_with_norm_arguments():
    g, n, d = _lib.pointer_array((P,)), _lib.size_array((16,)), _lib.dtype_array((0,))
    for norm, mx in ((None, 1.0), (P2 + 2, 1.0), (P2, -1.0), (P2, math.nan)):
        with pytest.raises(_lib.FlceError) as e:
            _lib.flce_clip_grads_with_norm(g, None, n, d, 1, mx, norm, None)
        assert e.value.status == INVALID


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    x, W = torch.zeros(4, 16), torch.zeros(8, 16)
    with pytest.raises(ValueError):
        F.flce_linear_forward(x, W)
    with pytest.raises(ValueError):
        F.flce_glu_forward(x, W, W)
    with pytest.raises(ValueError):
        F.flce_grad_norm([x])
    with pytest.raises(ValueError):
        F.flce_clip_grad_norm([], 1.0)
    with pytest.raises(ValueError):
        F.flce_linear_forward(x, W, activation="swish")
    with pytest.raises(ValueError):
        F.GatedFeedForward(16, 32, activation="swish")
    with pytest.raises(ValueError):
        F.flce_linear_backward(x, W, torch.zeros(4, 8), None, activation="relu")
    with pytest.raises(ValueError):
        F.flce_glu_backward(x, W, W, None, None, torch.zeros(4, 8))


def test_dense_in_any_order():
    t = torch.zeros(4, 6, 5)
    assert F._is_dense(t) and F._is_dense(t.permute(2, 0, 1)) and F._is_dense(torch.zeros(3, 1, 4).transpose(0, 2))
    assert not F._is_dense(t[:, ::2]) and not F._is_dense(t[:, :3]) and not F._is_dense(torch.zeros(1).expand(4))
    assert F._is_dense(torch.zeros(0, 3)) and F._is_dense(torch.zeros(()))
