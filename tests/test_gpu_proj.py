"""GPU: ssd_proj_fp8_fwd against the definition in 64 bits.

Bounds.  For y in fp32 a block's 128 products are exact and their sum fp32, at most one unit of 2^-23 of the sum of
magnitudes an addition; the blocks join by an fma each (2^-24), the scales' product is one rounding, and eight partial sums
join at the end: (256 + 2 blocks + 32) * 2^-24 of sum |a w| scales.  For y in bf16 the 8-bit matrix unit also cuts each of
eight products that it adds together at 2^-13 of the largest one's exponent: 7 * 2^-13 of the largest magnitudes' product for
every eight columns of K.  Then one rounding to the output's type."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV, U = "cuda", 2.0 ** -24
T = {"f32": torch.float32, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn


def make(M, N, K, seed=0):
    g = torch.Generator().manual_seed(seed + M + 3 * N + 7 * K)
    kb, nb = -(-K // 128), -(-N // 128)
    a, w = ((torch.randn(n, K, generator=g) * 60).clamp(-448, 448).to(E4M3) for n in (M, N))
    # scales that differ by thousands from block to block, negative and zero ones among them
    sa, sw = (torch.exp(torch.randn(n, kb, generator=g) * 2) * 0.01 for n in (M, nb))
    sa[::5, 0], sw[0, -1] = 0.0, -sw[0, -1]
    return dict(a=a, a_scale=sa, w=w, w_scale=sw)


def reference(d, t):
    """y in 64 bits, and the bound of its error before the last rounding."""
    K, N = d["a"].shape[1], d["w"].shape[0]
    wide = lambda s: s.double().repeat_interleave(128, 1)[:, :K]  # noqa: E731
    a, w = d["a"].double() * wide(d["a_scale"]), d["w"].double() * wide(d["w_scale"]).repeat_interleave(128, 0)[:N]
    mag = (256 + 2 * -(-K // 128) + 32) * U * (a.abs() @ w.abs().t())
    if t == "bf16":
        eight = lambda x: x.abs().reshape(x.shape[0], K // 8, 8).amax(-1)  # noqa: E731
        mag = mag + 7 * 2.0 ** -13 * (eight(a) @ eight(w).t())
    return a @ w.t(), mag


def verify(ssd, d, t, **kw):
    g = {n: v.to(DEV) for n, v in d.items()}
    y = ssd.ssd_proj_fp8_fwd(g["a"], g["a_scale"], g["w"], g["w_scale"], out_dtype=T[t], **kw)
    want, mag = reference(d, t)
    step = torch.finfo(T[t]).eps / 2
    err, lim = (y.double().cpu() - want).abs(), mag + step * (want.abs() + mag) + 1e-30
    assert y.dtype == T[t] and y.shape == want.shape and (err <= lim).all(), (float(err.max()), float((err / lim).max()), (err > lim).nonzero()[:4])
    return y


SIZES = [(1, 1, 16), (1, 16, 128), (3, 17, 144), (16, 128, 256), (17, 129, 1040), (32, 100, 512), (33, 300, 400), (64, 64, 4096),
         (65, 130, 2064), (100, 5, 16), (257, 128, 128), (300, 260, 1040), (513, 1000, 272), (129, 2000, 640),
         (260, 140, 4368), (300, 129, 2048), (257, 40, 2064), (520, 256, 6000)]


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_proj(gpu_lib, M, N, K, t):
    print(f"proj M={M} N={N} K={K} {t}", flush=True)
    verify(gpu_lib, make(M, N, K), t)


@pytest.mark.parametrize("M,N,K", [(3600, 3500, 272), (3585, 3600, 128), (4096, 4096, 144), (3600, 3500, 4384), (3585, 3600, 2064)])
def test_proj_of_many_tiles(gpu_lib, M, N, K):
    """Sizes at which the largest tiles are taken, full and cut, in every place of the launch order."""
    d = make(M, N, K)
    verify(gpu_lib, d, "bf16")


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("K", [128, 144, 256, 384, 400, 528, 656, 2048, 2064, 2192, 4368])
def test_proj_of_middling_sizes(gpu_lib, K, t):
    """Sizes at which the smallest tiles are taken, from one block to more than two sets of 16 scales, full and cut; the same
    from wider rows full of NaN."""
    for M, N in ((1000, 1000), (1024, 960)):
        d = make(M, N, K)
        want = verify(gpu_lib, d, t)
        g = {}
        for n in ("a", "w"):
            wide = torch.full((d[n].shape[0], K + 32), float("nan"), device=DEV).to(E4M3)
            wide.view(torch.uint8)[:, 16:16 + K] = d[n].to(DEV).view(torch.uint8)
            g[n] = wide[:, 16:16 + K]
        out = torch.full((M, N + 7), 7.0, dtype=T[t], device=DEV)
        y = gpu_lib.ssd_proj_fp8_fwd(g["a"], d["a_scale"].to(DEV), g["w"], d["w_scale"].to(DEV), y=out[:, 3:3 + N])
        assert torch.equal(y, want) and (out[:, :3] == 7).all() and (out[:, 3 + N:] == 7).all()


def test_proj_exact_sums(gpu_lib):
    """Small whole numbers and scales that are powers of two: every sum is exact, so is y."""
    g = torch.Generator().manual_seed(3)
    for M, N, K in ((5, 40, 384), (40, 200, 272), (300, 300, 656), (1000, 1000, 2064), (3600, 3600, 176)):
        kb = -(-K // 128)
        a, w = (torch.randint(-4, 5, (n, K), generator=g).float() for n in (M, N))
        sa, sw = 2.0 ** torch.randint(-2, 3, (M, kb), generator=g), 2.0 ** torch.randint(-2, 3, (-(-N // 128), kb), generator=g)
        ops = [v.to(DEV) for v in (a.to(E4M3), sa, w.to(E4M3), sw)]
        wide = lambda s: s.double().repeat_interleave(128, 1)[:, :K]  # noqa: E731
        want = (a.double() * wide(sa)) @ (w.double() * wide(sw).repeat_interleave(128, 0)[:N]).t()
        assert torch.equal(gpu_lib.ssd_proj_fp8_fwd(*ops, out_dtype=torch.float32).cpu().double(), want), (M, N, K)
        assert torch.equal(gpu_lib.ssd_proj_fp8_fwd(*ops).cpu(), want.float().to(torch.bfloat16)), (M, N, K)


def test_proj_strides(gpu_lib):
    """Operands in wider rows full of NaN, y as columns of wider rows on four elements and off them; what is beside stays."""
    for M, N, K in ((5, 70, 144), (200, 70, 272), (300, 200, 400), (3600, 3600, 144)):
        d = make(M, N, K)
        want = verify(gpu_lib, d, "bf16")
        g = {}
        for n in ("a", "w"):
            wide = torch.full((d[n].shape[0], K + 48), float("nan"), device=DEV).to(E4M3)
            wide.view(torch.uint8)[:, 16:16 + K] = d[n].to(DEV).view(torch.uint8)
            g[n] = wide[:, 16:16 + K]
            s = d[n + "_scale"]
            wide = torch.full((s.shape[0], s.shape[1] + 3), float("nan"), device=DEV)
            wide[:, 1:1 + s.shape[1]] = s.to(DEV)
            g[n + "_scale"] = wide[:, 1:1 + s.shape[1]]
        for lead, pad in ((4, 4), (3, 2), (1, 0)):
            out = torch.full((M, lead + N + pad), 7.0, dtype=torch.bfloat16, device=DEV)
            y = gpu_lib.ssd_proj_fp8_fwd(g["a"], g["a_scale"], g["w"], g["w_scale"], y=out[:, lead:lead + N])
            assert torch.equal(y, want) and (out[:, :lead] == 7).all() and (out[:, lead + N:] == 7).all()


def test_proj_nan_stays_in_its_row_and_column(gpu_lib):
    for M, N, K in ((5, 40, 272), (300, 300, 272), (1000, 1000, 272), (3600, 3600, 272)):
        d = {n: v.to(DEV) for n, v in make(M, N, K).items()}
        clean = gpu_lib.ssd_proj_fp8_fwd(d["a"], d["a_scale"], d["w"], d["w_scale"])
        d["a"].view(torch.uint8)[2, K - 1] = 0x7f
        d["w"].view(torch.uint8)[N - 3, K - 2] = 0xff
        y = gpu_lib.ssd_proj_fp8_fwd(d["a"], d["a_scale"], d["w"], d["w_scale"])
        assert torch.isnan(y[2]).all() and torch.isnan(y[:, N - 3]).all()
        y[2], y[:, N - 3] = clean[2], clean[:, N - 3]
        assert torch.equal(y, clean)


def test_proj_rows_do_not_depend_on_their_number(gpu_lib):
    """Within a kernel a row's bits are its own; more dimensions of rows are one."""
    d = {n: v.to(DEV) for n, v in make(16, 200, 1040).items()}
    y = gpu_lib.ssd_proj_fp8_fwd(d["a"], d["a_scale"], d["w"], d["w_scale"])
    for m in (0, 7, 15):
        assert torch.equal(gpu_lib.ssd_proj_fp8_fwd(d["a"][m:m + 1], d["a_scale"][m:m + 1], d["w"], d["w_scale"]), y[m:m + 1])
    y3 = gpu_lib.ssd_proj_fp8_fwd(d["a"].view(2, 8, 1040), d["a_scale"].view(2, 8, 9), d["w"], d["w_scale"])
    assert torch.equal(y3.view(16, 200), y)
    e = gpu_lib.ssd_proj_fp8_fwd(d["a"][:0], d["a_scale"][:0], d["w"], d["w_scale"])
    assert e.shape == (0, 200)


def test_proj_past_4g_bytes(gpu_lib):
    """Rows of a and of y that start past 2^32 bytes."""
    M, N, K, sa, sy = 1100, 40, 256, 4_194_304, 2_100_000
    d = make(M, N, K)
    want = verify(gpu_lib, d, "bf16")
    wide = torch.empty(M * sa, dtype=torch.uint8, device=DEV).view(M, sa)
    wide[:, 16:16 + K] = d["a"].to(DEV).view(torch.uint8)
    out = torch.empty(M * sy, dtype=torch.bfloat16, device=DEV).view(M, sy)
    y = gpu_lib.ssd_proj_fp8_fwd(wide[:, 16:16 + K].view(E4M3), d["a_scale"].to(DEV), d["w"].to(DEV), d["w_scale"].to(DEV), y=out[:, 8:8 + N])
    assert torch.equal(y.contiguous(), want)


def test_proj_on_streams_and_captured(gpu_lib):
    ssd = gpu_lib
    for M, N, K in ((4, 300, 528), (400, 300, 528)):
        sets = [{n: v.to(DEV) for n, v in make(M, N, K, seed=s).items()} for s in range(3)]
        call = lambda d, **kw: ssd.ssd_proj_fp8_fwd(d["a"], d["a_scale"], d["w"], d["w_scale"], **kw)  # noqa: E731
        want = [call(d) for d in sets]
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        got = call(sets[1], stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, want[1])
        g = {n: v.clone() for n, v in sets[0].items()}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = call(g)
        for k in (1, 2, 0):
            for n, v in sets[k].items():
                g[n].copy_(v)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want[k]) and torch.equal(call(sets[k]), want[k])
