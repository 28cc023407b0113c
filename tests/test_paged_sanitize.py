"""The paged operators' host checks under AddressSanitizer and
UndefinedBehaviorSanitizer, CPU only: tests/host/paged_validate_fuzz.cpp is built
with g++ together with csrc/paged/paged_validate.cpp and drives every checking
entry point with random, extreme and malformed arguments."""
import os
import shutil
import subprocess

import pytest

from test_host_sanitize import FLAGS, ROOT


def test_paged_checks_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    csrc = os.path.join(ROOT, "decode_gemv_elementwise_amd", "csrc", "paged")
    exe = str(tmp_path / "paged_validate_fuzz")
    r = subprocess.run([gxx, *FLAGS, "-I", os.path.join(ROOT, "include"), "-I", csrc,
                        os.path.join(ROOT, "tests", "host", "paged_validate_fuzz.cpp"),
                        os.path.join(csrc, "paged_validate.cpp"), "-o", exe], capture_output=True, text=True, timeout=300)
    if r.returncode != 0 and "sanitize" in r.stderr and ("cannot find" in r.stderr or "not supported" in r.stderr):
        pytest.skip("sanitizer runtime not available: " + r.stderr[-300:])
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe, "300000"], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-4000:])
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-4000:]
    assert r.stdout.startswith("ok 300000 iterations")
