"""The host side of the norm, the microscaled calls and the sampler under AddressSanitizer and
UndefinedBehaviorSanitizer: their boundary tests against a build of flce_api.hip whose launchers only return an error, so
that no kernel can run (CPU only; device code is not instrumented).
"""

import os
import re
import shlex
import subprocess
import sys
import tempfile

import pytest

sanitized = pytest.importorskip("test_boundary_sanitized")   # where the build's flags are
CSRC, HIPCC, ROOT, SAN, _runtime = (getattr(sanitized, name) for name in ("CSRC", "HIPCC", "ROOT", "SAN", "_runtime"))


@pytest.mark.timeout(300)
def test_tail_boundary_under_asan_and_ubsan():
    rt = _runtime()
    if not os.path.exists(HIPCC) or rt is None:
        pytest.skip("hipcc or the ASan runtime is not available")
    with tempfile.TemporaryDirectory(prefix="flce_san_") as tmp:
        stub = ['#include "layer_launch.hpp"', "namespace flce {"]
        for name in ("flce_launch.hpp", "layer_launch.hpp"):
            text = open(os.path.join(CSRC, name)).read()
            for d in re.findall(r"^(?:FLCE_WEAK )?(hipError_t launch_\w+\([^;]*?\));", text, re.M | re.S):
                stub.append(" ".join(d.split()) + " { return hipErrorNotSupported; }")
        assert sum("launch_" in line for line in stub) >= 20
        with open(os.path.join(tmp, "stub.cpp"), "w") as f:
            f.write("\n".join(stub + ["}", ""]))
        inc = f"-I{os.path.join(ROOT, 'include')} -I{CSRC}"
        cmds = [
            f"{HIPCC} --offload-arch=gfx950 -O1 -g -std=c++17 -fPIC -Xclang -target-feature -Xclang "
            f"-packed-fp32-ops {inc} -c {os.path.join(CSRC, 'flce_api.hip')} -o {tmp}/api.o {SAN}",
            f"{HIPCC} -O1 -std=c++17 -fPIC {inc} -c {tmp}/stub.cpp -o {tmp}/stub.o",
            f"{HIPCC} -shared -fPIC -o {tmp}/libflce_san.so {tmp}/api.o {tmp}/stub.o {SAN} -shared-libsan",
        ]
        for c in cmds:
            r = subprocess.run(shlex.split(c), capture_output=True, text=True)
            assert r.returncode == 0, r.stdout + r.stderr
        child = (
            "import sys\n"
            f"sys.path.insert(0, {ROOT!r})\n"
            "import lm_head_cross_flce_amd._lib as L\n"
            f"L.LIB_PATH = {tmp + '/libflce_san.so'!r}\n"
            "import pytest\n"
            "sys.exit(pytest.main(['-q', '-s', '-p', 'no:cacheprovider', '-k', 'not binding and not package', "
            f"{os.path.join(ROOT, 'tests', 'test_tail_boundary.py')!r}]))\n"
        )
        env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
                   UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
        r = subprocess.run([sys.executable, "-c", child], capture_output=True, text=True, env=env, cwd=ROOT)
        out = r.stdout + r.stderr
        assert r.returncode == 0 and "runtime error" not in out and "AddressSanitizer" not in out, out[-4000:]
        assert re.search(r"\d+ passed", out), out[-2000:]
