"""The host code of the operators on rows of logits and of the block norm seam under AddressSanitizer and
UndefinedBehaviorSanitizer (no GPU needed): ``tests/host_sanitizer/operators.cpp`` linked to the sanitizer build that
``tests/test_host_sanitizers.py`` makes of the library."""
import os
import subprocess

import pytest

from tests import test_host_sanitizers as H

DRIVER = os.path.join(H.ROOT, "tests", "host_sanitizer", "operators.cpp")


@pytest.mark.skipif(not (os.path.exists(H.HIPCC) and os.path.exists(H.CLANGXX)), reason="ROCm toolchain not found")
def test_operators_host_code_is_clean_under_asan_and_ubsan():
    H._build()
    drv = os.path.join(H.OUT, "operators_driver")
    r = subprocess.run([H.CLANGXX, "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer", "-I", H.INC, DRIVER, "-o", drv,
                        "-L", H.OUT, "-lpoet_sanitize", f"-Wl,-rpath,{H.OUT}"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ)
    env["ASAN_OPTIONS"] = "detect_leaks=0:abort_on_error=1:verify_asan_link_order=0"
    env["UBSAN_OPTIONS"] = "print_stacktrace=1:halt_on_error=1"
    r = subprocess.run([drv], capture_output=True, text=True, env=env, timeout=300)
    report = r.stdout + r.stderr
    assert r.returncode == 0, report[-6000:]
    assert "all checks passed" in r.stdout and "runtime error" not in report, report[-6000:]
