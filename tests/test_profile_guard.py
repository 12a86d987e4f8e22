"""The recorded figures of the loss's kernels are guarded by a hash of the loss's own sources (CPU)."""

import glob
import os
import re

import bench

CSRC = os.path.join(bench.ROOT, "lm_head_cross_flce_amd", "csrc")


def sources():
    return {os.path.basename(f): open(f).read() for f in glob.glob(os.path.join(CSRC, "*"))}


def test_other_operators_leave_the_hash_alone():
    src = sources()
    h = bench.kernel_source_hash(src)
    assert h == bench.kernel_source_hash()
    for name in src:
        changed = bench.kernel_source_hash({**src, name: src[name] + "\nint one_more;\n"})
        assert (changed == h) == name.startswith(("layer_", "grad_norm_")), name


def test_the_loss_is_compiled_from_no_other_operators_file():
    # flce_api.hip includes the other operators' entry points at its very end, behind the loss's
    src = sources()
    for name, text in src.items():
        if not name.startswith(bench.OTHER_OPERATORS) and name != "flce_api.hip":
            assert not re.search(r'#include "(layer_|grad_norm_)', text), name
    includes = re.findall(r'#include "(?:layer_|grad_norm_)\w+\.hpp"\n', src["flce_api.hip"])
    assert len(includes) == 2 and src["flce_api.hip"].endswith("".join(includes))
