"""Refusals of the norm, the microscaled calls and the sampler, without a GPU.

Every call carries one invalid argument that validation must catch before anything is enqueued; the placeholder
addresses are never dereferenced.
"""

import math
import os

import pytest
import torch

from lm_head_cross_flce_amd import _lib
from lm_head_cross_flce_amd import functional as F

# 64 MiB apart: no tensor of these calls reaches the next
X, R, Wt, Y, Hh, S, C, WS, D = (0x10000000 + (i << 26) for i in range(9))
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


def norm_fwd(**o):
    a = dict(x=X, residual=R, weight=Wt, N=100, H=4096, dtype=1, eps=1e-6, y=Y, h=Hh, rstd=S, stream=None)
    a.update(o)
    _lib.flce_rms_norm_forward(**a)


def norm_mx(**o):
    a = dict(x=X, residual=R, weight=Wt, N=100, H=4096, dtype=1, eps=1e-6, format=0, codes=C, scales=D, h=Hh, rstd=S,
             stream=None)
    a.update(o)
    _lib.flce_rms_norm_mx_forward(**a)


def norm_bwd(**o):
    a = dict(h=X, weight=Wt, rstd=S, dy=Y, dh=Hh, N=100, H=4096, dtype=1, dx=D, dweight=C, workspace=WS,
             workspace_bytes=BIG, stream=None)
    a.update(o)
    _lib.flce_rms_norm_backward(**a)


def quantize(**o):
    a = dict(x=X, R=100, C=1000, dtype=1, format=1, codes=C, scales=S, stream=None)
    a.update(o)
    _lib.flce_mx_quantize(**a)


def dequantize(**o):
    a = dict(codes=C, scales=S, R=100, C=1000, format=1, dtype=1, y=Y, stream=None)
    a.update(o)
    _lib.flce_mx_dequantize(**a)


def linear(**o):
    a = dict(x=X, x_scales=S, x_format=0, W=Wt, W_scales=D, b=C, residual=R, N=100, K=4096, F=256, dtype=1, activation=4,
             y=Y, workspace=WS, workspace_bytes=BIG, stream=None)
    a.update(o)
    _lib.flce_mx_linear(**a)


def sample(params=None, **o):
    a = dict(logits=X, u=S, N=4, V=1000, dtype=1, params=_lib.sampling(**(params or {})), tokens=Y, workspace=WS,
             workspace_bytes=BIG, stream=None)
    a.update(o)
    _lib.flce_sample(**a)


@pytest.mark.parametrize("fn", [norm_fwd, norm_mx, norm_bwd])
def test_norm_shapes_and_types(fn):
    refused(fn, INVALID, N=-1)
    refused(fn, INVALID, H=0)
    refused(fn, UNSUPPORTED, N=(1 << 30) + 1)
    refused(fn, UNSUPPORTED, H=(1 << 20) + 1)
    refused(fn, UNSUPPORTED, dtype=3)
    refused(fn, INVALID, weight=Wt + 1)
    for name, value in (("x", X), ("residual", R), ("h", Hh), ("y", Y), ("dy", Y), ("dh", Hh), ("dx", D)):
        if name in {norm_fwd: ("x", "residual", "h", "y"), norm_mx: ("x", "residual", "h"),
                    norm_bwd: ("h", "dy", "dh", "dx")}[fn]:
            refused(fn, INVALID, **{name: (X if name == "h" and fn is norm_bwd else value) + 8})


def test_norm_forward_arguments():
    for fn in (norm_fwd, norm_mx):
        refused(fn, INVALID, x=None)
        refused(fn, INVALID, rstd=S + 2)
        refused(fn, INVALID, residual=None)     # h would be x
        for eps in (-1e-6, math.nan, math.inf):
            refused(fn, INVALID, eps=eps)
        refused(fn, INVALID, h=X + 4096)        # over x, shifted
        refused(fn, INVALID, h=R + 4096)
        refused(fn, INVALID, rstd=X)
        refused(fn, INVALID, h=X, residual=X + 16)   # x, written in place, under the residual
    refused(norm_fwd, INVALID, y=None)
    refused(norm_fwd, INVALID, y=X)
    refused(norm_fwd, INVALID, y=R)
    refused(norm_fwd, INVALID, y=Hh)
    refused(norm_fwd, INVALID, y=Wt)
    refused(norm_mx, INVALID, format=2)
    refused(norm_mx, INVALID, format=-1)
    refused(norm_mx, INVALID, codes=None)
    refused(norm_mx, INVALID, scales=None)
    refused(norm_mx, INVALID, codes=C + 8)
    refused(norm_mx, INVALID, scales=D + 2)
    refused(norm_mx, INVALID, codes=X)
    refused(norm_mx, INVALID, scales=C)


def test_norm_backward_arguments():
    for name in ("h", "rstd", "dy"):
        refused(norm_bwd, INVALID, **{name: None})
    refused(norm_bwd, INVALID, dweight=C + 1)
    refused(norm_bwd, INVALID, dx=X)
    refused(norm_bwd, INVALID, dx=Y + 4096)
    refused(norm_bwd, INVALID, dx=Y, dh=Y + 4096)     # dy written in place, under dh
    refused(norm_bwd, INVALID, dweight=Wt)
    refused(norm_bwd, INVALID, workspace=D)
    need = _lib.flce_rms_norm_workspace_size(100, 4096, 1)
    assert need >= 4096 * 4
    refused(norm_bwd, TOO_SMALL, workspace_bytes=need - 1)
    refused(norm_bwd, INVALID, workspace=None)
    refused(norm_bwd, INVALID, workspace=WS + 8)
    refused(norm_bwd, INVALID, H=20000, dx=Y)         # long rows read dy again for dweight
    for bad in ((-1, 64), (4, 0)):
        with pytest.raises(_lib.FlceError):
            _lib.flce_rms_norm_workspace_size(*bad, 1)


@pytest.mark.parametrize("fn", [quantize, dequantize])
def test_convert_arguments(fn):
    refused(fn, INVALID, R=-1)
    refused(fn, INVALID, C=0)
    refused(fn, INVALID, format=2)
    refused(fn, UNSUPPORTED, dtype=3)
    refused(fn, UNSUPPORTED, C=(1 << 20) + 1)
    refused(fn, INVALID, codes=None)
    refused(fn, INVALID, scales=None)
    refused(fn, INVALID, codes=C + 8)
    refused(fn, INVALID, scales=S + 1)
    plain = "x" if fn is quantize else "y"
    refused(fn, INVALID, **{plain: None})
    refused(fn, INVALID, **{plain: X + 2})
    refused(fn, INVALID, **{plain: C})
    refused(fn, INVALID, **{plain: S - 1600})
    if fn is quantize:
        refused(fn, INVALID, scales=C)


def test_linear_arguments():
    refused(linear, INVALID, N=-1)
    refused(linear, INVALID, K=0)
    refused(linear, INVALID, F=0)
    refused(linear, INVALID, x_format=2)
    refused(linear, INVALID, activation=6)
    refused(linear, INVALID, activation=-1)
    refused(linear, UNSUPPORTED, dtype=3)
    refused(linear, UNSUPPORTED, K=(1 << 20) + 1)
    refused(linear, UNSUPPORTED, F=(1 << 20) + 1)
    refused(linear, UNSUPPORTED, N=1 << 30, F=1 << 20)
    for name, value, off in (("x", X, 8), ("x_scales", S, 2), ("W", Wt, 8), ("W_scales", D, 2), ("y", Y, 8)):
        refused(linear, INVALID, **{name: None})
        refused(linear, INVALID, **{name: value + off})
    refused(linear, INVALID, b=C + 1)
    refused(linear, INVALID, residual=R + 8)
    for over in (X, S, Wt, D, C, R + 256):
        refused(linear, INVALID, y=over)


def test_linear_workspace():
    # 100 x 256 outputs over K = 8192: few tiles, so K is split
    need = _lib.flce_mx_linear_workspace_size(100, 8192, 256, 0, 1)
    assert need > 0
    refused(linear, TOO_SMALL, K=8192, workspace_bytes=need - 1)
    refused(linear, INVALID, K=8192, workspace=None)
    refused(linear, INVALID, K=8192, workspace=WS + 8)
    refused(linear, INVALID, K=8192, workspace=Y)
    assert _lib.flce_mx_linear_workspace_size(8192, 4096, 12288, 0, 1) == 0
    assert _lib.flce_mx_linear_workspace_size(1, 4096, 128256, 0, 1) == 0
    assert _lib.flce_mx_linear_workspace_size(0, 4096, 64, 0, 1) == 0
    for bad in ((-1, 64, 64), (4, 0, 64), (4, 64, 0)):
        with pytest.raises(_lib.FlceError):
            _lib.flce_mx_linear_workspace_size(*bad, 0, 1)


def test_sample_arguments():
    refused(sample, INVALID, N=-1)
    refused(sample, INVALID, V=0)
    refused(sample, UNSUPPORTED, V=(1 << 30) + 1)
    refused(sample, UNSUPPORTED, N=1 << 22)
    refused(sample, UNSUPPORTED, N=1 << 12, V=1 << 26)
    refused(sample, UNSUPPORTED, dtype=3)
    with pytest.raises(_lib.FlceError):
        _lib.flce_sample(X, S, 4, 1000, 1, None, Y, WS, BIG, None)
    for name, value, off in (("logits", X, 8), ("u", S, 2), ("tokens", Y, 4)):
        refused(sample, INVALID, **{name: None})
        refused(sample, INVALID, **{name: value + off})
    refused(sample, INVALID, params=dict(temperatures=R + 2))
    refused(sample, INVALID, params=dict(top_ks=R + 4))
    refused(sample, INVALID, params=dict(top_ps=R + 2))
    refused(sample, INVALID, params=dict(min_ps=R + 2))
    refused(sample, INVALID, tokens=X)
    refused(sample, INVALID, tokens=S - 16)
    refused(sample, INVALID, params=dict(top_ks=Y))
    need = _lib.flce_sample_workspace_size(4, 128256, 1)
    assert need >= 4 * 128256 // 32 * 4
    refused(sample, TOO_SMALL, V=128256, workspace_bytes=need - 1)
    refused(sample, INVALID, V=128256, workspace=None)
    refused(sample, INVALID, V=128256, workspace=WS + 8)
    refused(sample, INVALID, V=128256, workspace=X)
    assert _lib.flce_sample_workspace_size(4, 1000, 1) == 0 and _lib.flce_sample_workspace_size(0, 128256, 1) == 0


def test_calls_without_rows_need_no_tensors():
    _lib.flce_rms_norm_forward(None, None, None, 0, 8, 1, 1e-6, None, None, None, None)
    _lib.flce_mx_quantize(None, 0, 8, 1, 1, None, None, None)
    _lib.flce_mx_linear(None, None, 0, Wt, D, None, None, 0, 64, 64, 1, 0, None, None, 0, None)
    _lib.flce_sample(None, None, 0, 8, 1, _lib.sampling(), None, None, 0, None)


def test_binding_refusals():
    x = torch.zeros(4, 16)
    codes, scales = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8)
    q = F.MXTensor(codes, scales, 16, "e4m3")
    assert q.shape == (4, 16)
    for call in (lambda: F.flce_rms_norm_forward(x), lambda: F.flce_rms_norm_mx_forward(x),
                 lambda: F.flce_rms_norm_backward(x, None, torch.zeros(4), x), lambda: F.flce_mx_quantize(x),
                 lambda: F.flce_mx_dequantize(q), lambda: F.flce_mx_linear(q, q),
                 lambda: F.flce_sample(x, torch.zeros(4)), lambda: F.flce_mx_quantize(x, "e5m2"),
                 lambda: F.flce_rms_norm_mx_forward(x, format="e3m2"),
                 lambda: F.flce_rms_norm_forward(torch.zeros(4)),
                 lambda: F.flce_mx_dequantize(q._replace(cols=200)),
                 lambda: F.flce_mx_dequantize(q._replace(format="e2m1")),
                 lambda: F.flce_mx_dequantize(q._replace(cols=0)),
                 lambda: F.fused_rms_norm(x, None, torch.zeros(4, 8)),
                 lambda: F.MXLinear(torch.nn.Linear(16, 8), activation="swish"),
                 lambda: F.flce_sample(torch.zeros(4), torch.zeros(4))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: F.flce_mx_dequantize(q._replace(codes=codes.float())),
                 lambda: F.flce_mx_dequantize(q, torch.float64)):
        with pytest.raises(TypeError):
            call()


def test_package_names():
    import lm_head_cross_flce_amd as pkg
    for name in ("flce_rms_norm_workspace_size", "flce_rms_norm_forward", "flce_rms_norm_mx_forward",
                 "flce_rms_norm_backward", "flce_mx_quantize", "flce_mx_dequantize", "flce_mx_linear_workspace_size",
                 "flce_mx_linear", "flce_sample_workspace_size", "flce_sample", "MXTensor", "fused_rms_norm", "RMSNorm", "MXLinear"):
        assert getattr(pkg, name) is getattr(F, name)
