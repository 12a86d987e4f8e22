"""Where the 256-row tile of the microscaled product finds its scales: host arithmetic, compiled and walked over every
row length, K part and step that a call can have, without a GPU.

A row has `bytes` scales, one to 32 columns.  Steps of 128 columns run in pairs from a part's first column k0 (a multiple of
256) to its end; four steps share a run of 16 bytes of the row.  Every read has to lie inside the run, the run inside the
row, and a step inside the row has to get its own four bytes.
"""

import os
import shlex
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "lm_head_cross_flce_amd", "csrc")
HIPCC = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc")

WALK = r"""
#include <cstdio>
#include "layer_launch.hpp"
int main() {
  long steps = 0, past = 0, wrong = 0;
  for (int Kp = 512; Kp <= 6144; Kp += 128) {
    const int bytes = Kp / flce::kMxBlock;
    for (int k0 = 0; k0 < Kp; k0 += 256)
      for (int kext = 512; kext <= Kp - k0; kext += 128)   // a part ends at a multiple of 256, or with the row
        if (kext % 256 == 0 || k0 + kext == Kp)
          for (int step = 0; step < 2 * ((kext + 255) / 256); ++step) {
            const int k = k0 + 128 * step, first = k0 + 512 * (step / 4);
            const int run = flce::mx_scale_run(first, bytes), at = flce::mx_scale_place(k, first, bytes);
            ++steps;
            past += k >= Kp;
            wrong += run < 0 || run + 16 > bytes || at < 0 || at + 4 > 16;
            wrong += k < Kp && run + at != k / flce::kMxBlock;
          }
  }
  std::printf("%ld %ld %ld\n", steps, past, wrong);
}
"""


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc is not available")
def test_every_step_reads_inside_its_run(tmp_path):
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(WALK)
    cmd = f"{HIPCC} -O1 -std=c++17 -I{os.path.join(ROOT, 'include')} -I{CSRC} {src} -o {exe}"
    r = subprocess.run(shlex.split(cmd), capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    steps, past, wrong = map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split())
    assert steps > 50_000 and past > 200 and wrong == 0
