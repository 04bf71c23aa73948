"""Which kernel of the 8-bit projection takes a size (no GPU): every kernel has sizes that test_gpu_proj_kernels.py runs, and every size
is taken by the kernel that it is there for."""
import os

import pytest

from tests.proj_sizes import SIZES

CODE = {"f32": 0, "bf16": 1}
INT_MAX = 0x7fffffff


@pytest.fixture(scope="module")
def ssd():
    import selective_state_space_14_amd as ssd
    if not os.path.exists(ssd.LIB_PATH):
        from selective_state_space_14_amd import build
        build.build(verbose=False)
    ssd.load()
    return ssd


def test_every_kernel_has_sizes():
    assert set(SIZES) == {("f32", 16), ("f32", 32), ("f32", 64), ("f32", 128)} | {("bf16", k) for k in (16, 32, 64, 128, 256)}
    for (t, rows), sizes in SIZES.items():
        blocks = [-(-k // 128) for _, _, k in sizes]
        assert min(blocks) == 1 and any(16 < b <= 32 for b in blocks) and max(blocks) > 32, (t, rows)
        assert any(m % rows for m, _, _ in sizes) and any(n % 16 for _, n, _ in sizes) and any(k % 128 for _, _, k in sizes), (t, rows)


@pytest.mark.parametrize("t,rows", list(SIZES))
def test_sizes_take_their_kernel(ssd, t, rows):
    for s in SIZES[t, rows]:
        assert ssd.ssd_proj_fp8_tile_rows(*s, CODE[t]) == rows, (s, t)


def test_no_kernel_for_sizes_that_are_refused(ssd):
    for s in ((0, 16, 16, 1), (-1, 16, 16, 1), (4, 0, 16, 1), (4, 16, 0, 1), (4, 16, 24, 1), (4, 16, 16, 2), (4, 16, 16, -1),
              (INT_MAX, INT_MAX, 16, 1), (INT_MAX, 16, 16, 1)):
        assert ssd.ssd_proj_fp8_tile_rows(*s) == 0, s
    # the largest that are not: a launch counts 2^32 threads
    for s in ((16777215 * 128, 128, 16, 1), (128, 16777215 * 128, 16, 0), (1, INT_MAX - 127, 4096, 1)):
        assert ssd.ssd_proj_fp8_tile_rows(*s) == 128, s
