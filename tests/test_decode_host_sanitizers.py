"""tests/test_decode_abi.py in a child process against the library whose host
code of the C ABI is built with AddressSanitizer and UndefinedBehaviorSanitizer
(no recovery). No GPU call is made."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_decode_abi_under_host_sanitizers():
    from mxfp8_decode_gemm_amd import build as b

    try:
        lib, runtime = b.build_host_sanitized(), b.host_asan_runtime()
    except RuntimeError as e:
        pytest.fail(f"host sanitizer build: {e}")
    # The interpreter itself is not instrumented: its allocations are not leak-checked.
    env = dict(os.environ, MXG_LIBRARY=lib, LD_PRELOAD=runtime,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_decode_abi.py"),
                        "-k", "not host_tensors"],  # that one imports torch
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and " passed" in out, out[-4000:]
    assert "ERROR: AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
