"""Outputs that share memory with another tensor of the call are refused, without a GPU.

Placeholder addresses, never dereferenced: every call here is refused.
"""

import os

import pytest

from lm_head_cross_flce_amd import _lib

N, H, F, DT = 100, 4096, 4096, 1   # bf16; F == H, so that every tensor could stand for another
MB = 1 << 20
STEP = 64 * MB                     # no tensor or workspace of these sizes is larger


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from lm_head_cross_flce_amd import build
        build.build()
    return _lib.load()


def places(names):
    return {n: STEP * (i + 1) for i, n in enumerate(names)}


def call(fn, names, act, **over):
    a = {**places(names), **over}
    glu = "glu" in fn.__name__
    sizes = (_lib.flce_glu_workspace_size(N, H, F, DT) if glu else _lib.flce_linear_workspace_size(N, H, F, DT, act))
    need = sizes["backward" in fn.__name__]
    assert 0 < need < STEP
    a.update(N=N, H=H, F=F, dtype=DT, activation=act, workspace_bytes=need, stream=None)
    return fn(**a)


NF, FH, NH = N * F * 2, F * H * 2, N * H * 2
LINEAR_FWD = dict(x=NH, W=FH, b=F * 2, residual=NF, y=NF, z=2 * NF, workspace=None)
LINEAR_BWD = dict(x=NH, W=FH, z=2 * NF, dy=NF, dx=NH, dW=FH, db=F * 2, workspace=None)
GLU_FWD = dict(x=NH, Wg=FH, Wu=FH, bg=F * 2, bu=F * 2, h=NF, g=2 * NF, u=2 * NF, workspace=None)
GLU_BWD = dict(x=NH, Wg=FH, Wu=FH, g=2 * NF, u=2 * NF, dh=NF, dx=NH, dWg=FH, dWu=FH, dbg=F * 2, dbu=F * 2, workspace=None)
WRITTEN = {"y", "z", "h", "dx", "dW", "db", "dWg", "dWu", "dbg", "dbu", "workspace"}
CALLS = [(_lib.flce_linear_forward, LINEAR_FWD, WRITTEN), (_lib.flce_linear_backward, LINEAR_BWD, WRITTEN - {"z"}),
         (_lib.flce_glu_forward, GLU_FWD, WRITTEN | {"g", "u"}), (_lib.flce_glu_backward, GLU_BWD, WRITTEN)]


@pytest.mark.parametrize("fn,sizes,written", CALLS, ids=lambda v: getattr(v, "__name__", ""))
def test_shared_memory_is_refused(fn, sizes, written):
    at = places(sizes)
    for out in sizes:
        if out not in written:
            continue
        for other in sizes:
            if other == out or {out, other} == {"y", "residual"}:
                continue
            last = (sizes[other] or 4096) - 16   # within the other's last 16 bytes, and at its very start
            for shift in (0, last // 16 * 16):
                with pytest.raises(_lib.FlceError) as e:
                    call(fn, sizes, 4, **{out: at[other] + shift})
                assert e.value.status == _lib.FLCE_ERR_INVALID_ARGUMENT, (out, other, shift)


def test_residual_may_be_the_output_but_not_overlap_it():
    at = places(LINEAR_FWD)
    for shift in (16, -16, NF - 16):
        with pytest.raises(_lib.FlceError) as e:
            call(_lib.flce_linear_forward, LINEAR_FWD, 4, residual=at["y"] + shift)
        assert e.value.status == _lib.FLCE_ERR_INVALID_ARGUMENT, shift
    # the residual itself as the output, over x: refused for x
    with pytest.raises(_lib.FlceError) as e:
        call(_lib.flce_linear_forward, LINEAR_FWD, 4, residual=at["x"], y=at["x"])
    assert e.value.status == _lib.FLCE_ERR_INVALID_ARGUMENT
