"""Argument validation of the entry points around the cache of keys and values under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): tests/sanitize/kv_checks.cpp against a sanitized build of
abi.cpp's host code, as tests/test_abi_sanitized.py does for the other calls."""
import os
import subprocess
import tempfile

import pytest

from precision_quantized_linear_amd import build as B
from test_abi_sanitized import ROOT, SAN, _objects

DRIVER = os.path.join(ROOT, "tests", "sanitize", "kv_checks.cpp")


@pytest.mark.skipif(not os.path.exists(B.hipcc()), reason="hipcc is not installed")
def test_kv_validation_under_asan_and_ubsan():
    objs = _objects()
    with tempfile.TemporaryDirectory() as tmp:
        flags = ["-O1", "-g", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", B.CSRC,
                 "-Wno-unused-command-line-argument"]
        abi_o, drv_o, exe = (os.path.join(tmp, n) for n in ("abi_san.o", "drv.o", "kv_checks"))
        for cmd in ([B.hipcc(), *flags, f"--offload-arch={B.ARCH}", *SAN, "-x", "hip", "-c",
                     os.path.join(B.CSRC, "abi.cpp"), "-o", abi_o],
                    [B.hipcc(), *flags, *SAN, "-x", "c++", "-c", DRIVER, "-o", drv_o],
                    [B.hipcc(), f"--offload-arch={B.ARCH}", *SAN, drv_o, abi_o, *objs, "-o", exe]):
            r = subprocess.run(cmd, capture_output=True, text=True)
            assert r.returncode == 0, f"{' '.join(cmd[:3])} ...: {r.stderr[-2000:]}"
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
        r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
        out = r.stdout + r.stderr
        assert r.returncode == 0 and "ok: 0 failures" in r.stdout, out[-4000:]
        assert "runtime error" not in out and "AddressSanitizer" not in out, out[-4000:]
