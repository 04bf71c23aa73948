"""The kernels of sources that are compiled with flags of their own run without scratch memory as they are built.

test_kernel_resources.py compiles every source with the flags they share; a source's own (accumulators in vector registers)
change its register counts, so those are compiled again here as the library is.  No GPU is needed."""
from __future__ import annotations

import concurrent.futures
import os
import re
import shutil
import subprocess

import pytest

from selective_state_space_14_amd import build as hip_build

OWN = sorted(hip_build.EXTRA_CFLAGS)


def _kernel_scratch(src: str, out_dir: str) -> dict:
    asm = os.path.join(out_dir, src + ".s")
    flags = [f for f in hip_build.cflags(src) if f not in ("-fPIC", "-Wall")]
    cmd = [hip_build.HIPCC, *flags, "--cuda-device-only", "-S", os.path.join(hip_build.CSRC, src), "-o", asm]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, f"hipcc failed on {src}:\n{r.stderr[-2000:]}"
    out = {}
    for block in re.split(r"\n  - \.", open(asm).read().split("amdhsa.kernels:", 1)[1]):
        name = re.search(r"\.name:\s+(\S+)", block)
        size = re.search(r"\.private_segment_fixed_size:\s+(\d+)", block)
        if name and size:
            out[name.group(1)] = int(size.group(1))
    return out


def test_the_build_uses_these_flags(monkeypatch, tmp_path):
    """What _compile runs is what is checked here."""
    seen = {}

    def run(cmd, **kw):
        seen[os.path.basename(cmd[cmd.index("-c") + 1])] = cmd
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(hip_build.subprocess, "run", run)
    for src in hip_build.SOURCES:
        hip_build._compile(src, str(tmp_path))
        flags = hip_build.cflags(src)
        assert seen[src][1:1 + len(flags)] == flags and seen[src][1 + len(flags)] == "-c", seen[src]
        assert (len(flags) > len(hip_build.CFLAGS)) == (src in OWN)


@pytest.mark.skipif(not (os.path.exists(hip_build.HIPCC) or shutil.which("hipcc")), reason="hipcc not found")
def test_no_kernel_uses_scratch_as_built(tmp_path):
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(OWN)) as ex:
        kernels = {k: v for d in ex.map(lambda s: _kernel_scratch(s, str(tmp_path)), OWN) for k, v in d.items()}
    # every instantiation of the delta rule's kernels was read
    for name, count in (("prep", 4), ("chain", 4), ("join", 2), ("scan", 2), ("back", 2), ("reverse", 1), ("grad", 2)):
        for n in (32, 64, 128):
            of = [k for k in kernels if re.search(rf"ssd_delta_{name}_kernelI\w*Li{n}E", k)]
            assert len(of) == count, (name, n, of)
    spilled = {k: v for k, v in kernels.items() if v != 0}
    assert not spilled, spilled
