"""The argument checks of tests/test_abi_rows.py again, on the build whose host code is instrumented with AddressSanitizer and
UndefinedBehaviorSanitizer.  No GPU: no call in them launches anything."""
import os
import subprocess
import sys

import pytest

from bit_nf4_quantized_11_amd import build
from test_abi_sanitized import ROOT, _asan_runtime


def test_abi_rows_under_address_and_ub_sanitizers():
    rt = _asan_runtime()
    if rt is None:
        pytest.skip("no AddressSanitizer runtime in this toolchain")
    env = dict(os.environ)
    env["QLORA_LIB"] = build.build(sanitize=True)
    env["LD_PRELOAD"] = rt + (":" + env["LD_PRELOAD"] if env.get("LD_PRELOAD") else "")
    env["ASAN_OPTIONS"] = "detect_leaks=0:abort_on_error=1"
    env["UBSAN_OPTIONS"] = "print_stacktrace=1:halt_on_error=1"
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "not gpu",
                        os.path.join(ROOT, "tests", "test_abi_rows.py")], cwd=ROOT, env=env, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
    assert "passed" in r.stdout
