"""The delta rule's and the norm's size checks at the ends of their integers, without a GPU: refused on the host with a
message, under AddressSanitizer and UndefinedBehaviorSanitizer too (no product of sizes may overflow)."""
import os
import subprocess
import sys

import pytest

from tests.test_abi_delta_norm import bwd, fwd, lib, norm, refused, step  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MOST = 2 ** 31 - 1
HUGE = [dict(B=MOST, H=65536, L=1 << 30), dict(B=MOST, H=65536, L=1), dict(B=MOST, H=MOST, G=1, L=1 << 30),
        dict(B=1 << 20, H=1 << 20, L=1 << 30), dict(B=1 << 24, H=8, L=1 << 30), dict(B=MOST, H=MOST, G=1, L=0)]


@pytest.mark.parametrize("over", HUGE)
def test_delta_calls_refuse_more_heads_than_a_grid_holds(lib, over):  # noqa: F811
    for call in (fwd, bwd) + ((step,) if over["L"] == 1 else ()):
        refused(lib, call(lib, over), 2, "is too large")


@pytest.mark.parametrize("over", HUGE + [dict(B=1, H=1, L=MOST), dict(B=1, H=8, L=(1 << 30) + 1)])
def test_delta_sizes_that_calls_refuse_need_no_workspace(lib, over):  # noqa: F811
    for size in (lib.ssd_delta_scan_workspace_size, lib.ssd_delta_scan_bwd_workspace_size):
        for dtype in (0, 1):
            assert size(over["B"], over["L"], over["H"], 64, 64, 1, dtype) == 0


def test_norm_sizes(lib):  # noqa: F811
    refused(lib, norm(lib, True, dict(R=(1 << 62) + 1, groups=MOST)), 2, "are too many")
    refused(lib, norm(lib, False, dict(R=1 << 31, groups=1)), 2, "are too many")
    size = lib.ssd_norm_bwd_workspace_size
    assert size((1 << 62) + 1, MOST, 64) == size(1 << 40, 1, 64) == size(1 << 20, 1, 64) > 0


def test_under_host_asan_ubsan():
    from selective_state_space_14_amd import build
    if os.environ.get("SSD_LIBRARY"):
        pytest.skip("this is the sanitized run")
    try:
        runtime = build.host_sanitizer_runtime()
    except (RuntimeError, OSError) as e:
        pytest.skip(f"no ASan runtime: {e}")
    lib = build.build_host_sanitized(verbose=False)
    env = dict(os.environ, LD_PRELOAD=runtime, SSD_LIBRARY=lib, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    files = [os.path.join(ROOT, "tests", f) for f in ("test_abi_delta_norm.py", "test_abi_delta_norm_sizes.py")]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", *files], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=600)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0, tail
    assert "ERROR: AddressSanitizer" not in r.stderr and "runtime error:" not in r.stderr, tail
    assert " passed" in r.stdout, tail
