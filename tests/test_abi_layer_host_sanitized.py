"""The refusals of tests/test_abi_layer.py against a library whose host code is under AddressSanitizer and
UndefinedBehaviorSanitizer, in a child process.  No GPU is needed."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_layer_checks_under_host_asan_ubsan():
    from selective_state_space_14_amd import build
    try:
        runtime = build.host_sanitizer_runtime()
    except (RuntimeError, OSError) as e:
        pytest.skip(f"no ASan runtime: {e}")
    env = dict(os.environ, LD_PRELOAD=runtime, SSD_LIBRARY=build.build_host_sanitized(verbose=False),
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_abi_layer.py")], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0 and " passed" in r.stdout, tail
    assert "ERROR: AddressSanitizer" not in r.stderr and "runtime error:" not in r.stderr, tail
