"""The choice of tiles and K splits of the feed-forward operators, through the workspaces it asks for (CPU)."""

import math
import random

import pytest

from lm_head_cross_flce_amd import _lib


def backward_bytes(op, N, H, F, dtype):
    return (_lib.flce_glu_workspace_size(N, H, F, dtype) if op == "glu"
            else _lib.flce_linear_workspace_size(N, H, F, dtype, 4))[1]


@pytest.mark.parametrize("op", ["linear", "glu"])
def test_both_gradient_products_take_one_tile(monkeypatch, op):
    # float32 has two sizes of output tile, and the two gradient products share a launch and with it a size: the
    # splits, which the workspace holds sums for, are then those of one size for both products.  A size that one
    # product chose with a split that was costed for the other size asks for a workspace of neither.
    rng = random.Random(5)
    for _ in range(1500):
        N, H, F = (max(1, round(math.exp(rng.uniform(math.log(a), math.log(b)))))
                   for a, b in ((1, 8192), (8, 4096), (16, 8192)))
        monkeypatch.delenv("FLCE_DEBUG_LAYER_TILE", raising=False)
        got = backward_bytes(op, N, H, F, 0)
        want = set()
        for tile in ("2", "4"):
            monkeypatch.setenv("FLCE_DEBUG_LAYER_TILE", tile)
            want.add(backward_bytes(op, N, H, F, 0))
        assert got in want, (N, H, F, got, want)


def test_unknown_forced_tiles_are_ignored(monkeypatch):
    shapes = [(N, H, F) for N in (1, 5, 70, 517, 1037) for H in (72, 1000) for F in (40, 2731)]

    def sizes():
        return [f(*s, d, *a) for s in shapes for d in (0, 1, 2)
                for f, a in ((_lib.flce_linear_workspace_size, (4,)), (_lib.flce_glu_workspace_size, ()))]

    monkeypatch.delenv("FLCE_DEBUG_LAYER_TILE", raising=False)
    free = sizes()
    for value in ("", "0", "3", "16", "-4", "tile"):
        monkeypatch.setenv("FLCE_DEBUG_LAYER_TILE", value)
        assert sizes() == free, value
    monkeypatch.setenv("FLCE_DEBUG_LAYER_TILE", "4")
    assert sizes() != free


def test_the_package_names_the_size_queries():
    import torch

    import lm_head_cross_flce_amd as pkg
    assert pkg.flce_linear_workspace_size(70, 264, 100, torch.bfloat16, "gelu") == _lib.flce_linear_workspace_size(
        70, 264, 100, 1, 2)
    assert pkg.flce_glu_workspace_size(70, 264, 100, torch.float32) == _lib.flce_glu_workspace_size(70, 264, 100, 0)
