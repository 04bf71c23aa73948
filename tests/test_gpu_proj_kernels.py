"""GPU: every kernel of ssd_proj_fp8_fwd, by name, against the definition in 64 bits: ordinary values, operands in wider rows full of
NaN, sums that are exact, NaN of one row and column, and rows that do not depend on their number.  Bounds as in test_gpu_proj.py."""
import pytest
import torch

from tests.proj_sizes import SIZES
from tests.test_gpu_proj import DEV, E4M3, T, make, reference

pytestmark = pytest.mark.gpu

CODE = {"f32": 0, "bf16": 1}
CASES = [(t, rows, *s) for (t, rows), sizes in SIZES.items() for s in sizes]


def call(ssd, d, **kw):
    return ssd.ssd_proj_fp8_fwd(d["a"], d["a_scale"], d["w"], d["w_scale"], **kw)


def inside(v, lead, pad):
    """v as columns of wider rows that are NaN."""
    wide = torch.full((v.shape[0], lead + v.shape[1] + pad), float("nan"), device=DEV).to(v.dtype)
    raw = torch.uint8 if v.dtype == E4M3 else v.dtype
    wide.view(raw)[:, lead:lead + v.shape[1]] = v.view(raw)
    return wide[:, lead:lead + v.shape[1]]


@pytest.mark.parametrize("t,rows,M,N,K", CASES)
def test_proj_kernel(gpu_lib, t, rows, M, N, K):
    assert gpu_lib.ssd_proj_fp8_tile_rows(M, N, K, CODE[t]) == rows
    print(f"proj {t} {rows} M={M} N={N} K={K}", flush=True)
    d = {n: v.to(DEV) for n, v in make(M, N, K).items()}
    y = call(gpu_lib, d, out_dtype=T[t])
    want, mag = reference(d, t)
    err, lim = (y.double() - want).abs(), mag + torch.finfo(T[t]).eps / 2 * (want.abs() + mag) + 1e-30
    assert y.dtype == T[t] and y.shape == want.shape and (err <= lim).all(), (float((err / lim).max()), (err > lim).nonzero()[:4])
    del want, mag, err, lim
    # wider rows, and y as columns off four elements: the same bits, and what is beside y stays
    g = {n: inside(v, 16 if v.dtype == E4M3 else 1, 32 if v.dtype == E4M3 else 2) for n, v in d.items()}
    out = torch.full((M, N + 7), 7.0, dtype=T[t], device=DEV)
    assert torch.equal(call(gpu_lib, g, y=out[:, 3:3 + N]), y) and (out[:, :3] == 7).all() and (out[:, 3 + N:] == 7).all()
    # NaN of one row of a, near its end, and of one of w
    m, n = M * 2 // 3, N - 3
    d["a"].view(torch.uint8)[m, K - 1] = 0x7f
    d["w"].view(torch.uint8)[n, K - 2] = 0xff
    again = call(gpu_lib, d, out_dtype=T[t])
    assert torch.isnan(again[m]).all() and torch.isnan(again[:, n]).all()
    again[m], again[:, n] = y[m], y[:, n]
    assert torch.equal(again, y)


@pytest.mark.parametrize("t,rows,M,N,K", CASES)
def test_proj_kernel_exact_sums(gpu_lib, t, rows, M, N, K):
    """Small whole numbers and scales that are powers of two: every sum is exact, so is y (at most 16 * 16 * 4368 = 2^20.1 in
    steps of 2^-4, and of random signs, far below 2^24 steps)."""
    print(f"proj exact {t} {rows} M={M} N={N} K={K}", flush=True)
    g = torch.Generator().manual_seed(M + N + K)
    kb = -(-K // 128)
    a, w = (torch.randint(-4, 5, (n, K), generator=g).float().to(DEV) for n in (M, N))
    sa, sw = (2.0 ** torch.randint(-2, 3, (n, kb), generator=g) for n in (M, -(-N // 128)))
    sa, sw = sa.to(DEV), sw.to(DEV)
    wide = lambda s: s.double().repeat_interleave(128, 1)[:, :K]  # noqa: E731
    want = (a.double() * wide(sa)) @ (w.double() * wide(sw).repeat_interleave(128, 0)[:N]).t()
    y = gpu_lib.ssd_proj_fp8_fwd(a.to(E4M3), sa, w.to(E4M3), sw, out_dtype=T[t])
    assert gpu_lib.ssd_proj_fp8_tile_rows(M, N, K, CODE[t]) == rows and torch.equal(y, want.float().to(T[t]))


@pytest.mark.parametrize("t,rows", list(SIZES))
def test_proj_rows_do_not_depend_on_m_within_a_kernel(gpu_lib, t, rows):
    """The first rows of a larger call, where the same kernel takes both."""
    for M, N, K in SIZES[t, rows]:
        fewer = next((m for m in (M - 1, M - rows, M - 5) if m > 0 and gpu_lib.ssd_proj_fp8_tile_rows(m, N, K, CODE[t]) == rows), None)
        if fewer is None:
            continue
        print(f"proj rows {t} {rows} M={M} {fewer} N={N} K={K}", flush=True)
        d = {n: v.to(DEV) for n, v in make(M, N, K).items()}
        part = {**d, "a": d["a"][:fewer], "a_scale": d["a_scale"][:fewer]}
        assert torch.equal(call(gpu_lib, part, out_dtype=T[t]), call(gpu_lib, d, out_dtype=T[t])[:fewer]), (M, N, K)
