"""The tile schedule of the grouped products on the host under UndefinedBehaviorSanitizer (CPU only):
tests/sanitize/moe_tiles.cpp, built with the functions that the kernel itself calls."""
import os
import subprocess
import tempfile

import pytest

from precision_quantized_linear_amd import build as B
from test_abi_sanitized import ROOT, SAN

DRIVER = os.path.join(ROOT, "tests", "sanitize", "moe_tiles.cpp")


@pytest.mark.skipif(not os.path.exists(B.hipcc()), reason="hipcc is not installed")
def test_tiles_stay_inside_the_rows():
    with tempfile.TemporaryDirectory() as tmp:
        exe = os.path.join(tmp, "moe_tiles")
        cmd = [B.hipcc(), "-O1", "-g", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", B.CSRC,
               "-Wno-unused-command-line-argument", f"--offload-arch={B.ARCH}", *SAN, "-x", "hip", DRIVER, "-o", exe]
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
        r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
        out = r.stdout + r.stderr
        assert r.returncode == 0 and "ok: 0 failures" in r.stdout, out[-4000:]
        assert "runtime error" not in out and "AddressSanitizer" not in out, out[-4000:]
