"""The norm and the workspace of a clipping call share memory with no tensor of it (CPU; nothing is launched).

Placeholder addresses, never dereferenced: every call here is refused.
"""

import os

import pytest

from lm_head_cross_flce_amd import _lib

G, O, WS, NORM = 0x100000, 0x200000, 0x300000, 0x400000   # a gradient, its output, workspace, norm
COUNT, N = 1, 4096                                          # float32: 16 KB each


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from lm_head_cross_flce_amd import build
        build.build()
    return _lib.load()


def arrays(out):
    return (_lib.pointer_array([G]), _lib.pointer_array([O]) if out else None, _lib.size_array([N]),
            _lib.dtype_array([0]))


def refused(fn, *args):
    with pytest.raises(_lib.FlceError) as e:
        fn(*args)
    assert e.value.status == _lib.FLCE_ERR_INVALID_ARGUMENT


def clip(out, norm=NORM, workspace=WS):
    g, o, n, d = arrays(out)
    _lib.flce_clip_grad_norm(g, o, n, d, COUNT, 1.0, 2.0, norm, workspace, _lib.flce_grad_norm_workspace_size(COUNT), None)


def norm_of(norm=NORM, workspace=WS):
    g, _, n, d = arrays(False)
    _lib.flce_grad_norm(g, n, d, COUNT, 2.0, norm, workspace, _lib.flce_grad_norm_workspace_size(COUNT), None)


def by_given(out, norm):
    g, o, n, d = arrays(out)
    _lib.flce_clip_grads_with_norm(g, o, n, d, COUNT, 1.0, norm, None)


@pytest.mark.parametrize("out", [False, True])
def test_the_written_norm(out):
    for at in (G, G + 4 * N - 4, WS, *((O, O + 4 * N - 4) if out else ())):
        refused(clip, out, at)


@pytest.mark.parametrize("out", [False, True])
def test_the_workspace(out):
    size = _lib.flce_grad_norm_workspace_size(COUNT)
    for at in (G, G + 4 * N - 16, G - size + 16, *((O, O - size + 16) if out else ())):
        refused(clip, out, NORM, at)


def test_the_norm_alone():
    size = _lib.flce_grad_norm_workspace_size(COUNT)
    for at in (G, G + 4 * N - 4, WS, WS + size - 4):
        refused(norm_of, at)
    for at in (G, G + 4 * N - 16, G - size + 16):
        refused(norm_of, NORM, at)


def test_a_given_norm_that_the_call_would_scale():
    # some workgroups would read it before it is scaled, some after
    for at in (G, G + 4 * N - 4):
        refused(by_given, False, at)
    for at in (O, O + 4 * N - 4):
        refused(by_given, True, at)
