"""The build's check of matrix instructions' waits: on listings with and without the mistake, and on compiled code (never
run)."""

import os
import subprocess

import pytest

from lm_head_cross_flce_amd import build, matrix_waits

MFMA = "v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[8:11], a[0:3]"
SCALED = "v_mfma_scale_f32_16x16x128_f8f6f4 a[0:3], v[4:7], v[8:15], a[0:3], v20, v21 op_sel_hi:[0,0,0] cbsz:4"


def listing(*lines):
    """Lines of a function f at 0x100, 4 bytes each; `-> n` ends a branch to line n."""
    out = ["0000000000000100 <f>:"]
    for i, line in enumerate(lines):
        text, _, to = line.partition(" -> ")
        out.append(f"\t{text:60s}// {0x100 + 4 * i:012X}: 00000000" + (f" <f+{4 * int(to):#x}>" if to else ""))
    return "\n".join(out)


@pytest.mark.parametrize("before,bad", [
    (["v_mov_b32_e32 v5, v40"], True),
    (["v_mov_b32_e32 v5, v40", "s_nop 0"], True),
    (["v_mov_b32_e32 v5, v40", "s_nop 1"], False),
    (["v_mov_b32_e32 v5, v40", "s_add_i32 s0, s0, 1", "ds_read_b128 v[60:63], v64"], False),
    (["v_mov_b32_e32 v12, v40"], False),
    (["v_mov_b64_e32 v[6:7], v[40:41]"], True),
    (["v_accvgpr_write_b32 a2, v40", "s_nop 0"], True),
    (["v_accvgpr_read_b32 v40, a2"], False),
    (["v_readlane_b32 s4, v5, 3"], False),
    (["v_writelane_b32 v9, s4, 3"], True),
    (["v_swap_b32 v40, v10"], True),
    (["ds_read_b128 v[4:7], v64", "s_waitcnt lgkmcnt(0)"], False),
    (["v_cmpx_lt_i32_e32 v40, v41", "s_nop 2"], True),
    (["v_cmpx_lt_i32_e32 v40, v41", "s_nop 3"], False),
    ([MFMA.replace("a[0:3]", "a[4:7]")], False),
])
def test_what_comes_before(before, bad):
    count, found = matrix_waits.too_soon(listing(*before, MFMA, "s_endpgm"))
    assert count == 1 + sum("mfma" in b for b in before) and bool(found) == bad


@pytest.mark.parametrize("reg,bad", [("v20", True), ("v21", True), ("v15", True), ("v16", False), ("v22", False)])
def test_scales_are_operands(reg, bad):
    assert bool(matrix_waits.too_soon(listing(f"v_bfe_u32 {reg}, v40, 8, 8", SCALED, "s_endpgm"))[1]) == bad


def test_every_way_to_an_instruction():
    # a loop whose last line writes the operand that its first one reads
    loop = listing("s_nop 7", MFMA, "s_nop 7", "v_mov_b32_e32 v5, v40", "s_cbranch_scc1 65532 -> 1", "s_endpgm")
    assert matrix_waits.too_soon(loop)[1]
    waits = listing("s_nop 7", MFMA, "s_nop 7", "v_mov_b32_e32 v5, v40", "s_nop 0", "s_cbranch_scc1 65532 -> 1", "s_endpgm")
    assert not matrix_waits.too_soon(waits)[1]
    # a branch around the write, and one that never falls through to the instruction
    assert matrix_waits.too_soon(listing("s_cbranch_scc1 1 -> 2", "v_mov_b32_e32 v5, v40", MFMA, "s_endpgm"))[1]
    skipped = listing("s_branch 2 -> 3", "v_mov_b32_e32 v5, v40", "s_branch 1 -> 4", MFMA, "s_endpgm")
    assert not matrix_waits.too_soon(skipped)[1]


SOURCE = r"""
#include <hip/hip_runtime.h>
typedef float f4 __attribute__((ext_vector_type(4)));
typedef unsigned u4 __attribute__((ext_vector_type(4)));
__global__ void k(const u4* a, f4* c) {
  const u4 x = a[threadIdx.x];
  u4 y = x * 3u;                  // written by vector instructions, just before
  f4 z = {0.f, 0.f, 0.f, 0.f};
  asm volatile("WAIT v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0\n\ts_nop 15" : "+a"(z) : "v"(x), "v"(y));
  c[threadIdx.x] = z;
}
"""


@pytest.mark.skipif(not os.path.exists(build.hipcc()), reason="hipcc is not available")
@pytest.mark.parametrize("wait", ["", "s_nop 1\\n\\t"])
def test_compiled_code(tmp_path, wait):
    src, obj = tmp_path / "k.hip", tmp_path / "k.o"
    src.write_text(SOURCE.replace("WAIT ", wait))
    r = subprocess.run([build.hipcc()] + build.common_flags() + ["-c", str(src), "-o", str(obj)], capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stderr
    if wait:
        assert matrix_waits.check(str(obj)) == 1
    else:
        with pytest.raises(RuntimeError, match="too soon"):
            matrix_waits.check(str(obj))
