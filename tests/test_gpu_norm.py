"""GPU: ssd_norm_fwd and ssd_norm_bwd against the definition in 64 bits.

Bounds.  A row's fp32 sums are trees of at most 32 terms in a thread and 10 levels above, so a statistic is off by at
most 42 * 2^-24 of its sum of magnitudes; with the few roundings of every other step (each 2^-24, the hardware exp2 and
reciprocal 2^-23) 64 * 2^-24 covers one pass over them.  A centred row x - mean inherits the mean's error, relative to
mean|x|.  Each output is then rounded once to its type, by at most eps / 2 of itself.  Weight gradients add, for each
column, at most R / (rows a step) terms in order: 64 + R of 2^-24 of the sum of magnitudes."""
import pytest
import torch

from tests import delta_ref as ref

pytestmark = pytest.mark.gpu

DEV, U = "cuda", 2.0 ** -24
T = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(R, W, xt, t, bias=True, gate=False, seed=0, offset=0.5):
    g = torch.Generator().manual_seed(seed + 31 * W + R)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=(r(R, W) * 2 + offset).to(T[xt]), weight=1 + 0.3 * r(W), bias=0.3 * r(W) if bias else None,
                z=r(R, W).to(T[t]) if gate else None, gy=r(R, W).to(T[t]))


def up(d):
    return {n: None if v is None else v.to(DEV) for n, v in d.items()}


def half_step(t):
    return torch.finfo(T[t]).eps / 2


def hat_parts(d, rms):
    x = d["x"].double()
    c = x if rms else x - x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5)
    n = c * rstd
    off = 64 * U * (2 * n.abs() + (0.0 if rms else 1.0) * x.abs().mean(-1, keepdim=True) * rstd)   # error of n
    return n, rstd, off


def check_fwd(ssd, d, t, rms, **kw):
    g = up(d)
    y = ssd.ssd_norm_fwd(g["x"], g["weight"], bias=g["bias"], z=g["z"], rms=rms, out_dtype=T[t], **kw)
    want = ref.norm(d["x"], d["weight"], d["bias"], d["z"], rms)
    n, _, off = hat_parts(d, rms)
    w = torch.ones(()) if d["weight"] is None else d["weight"].double().abs()
    mag = off * w + 4 * U * (n.abs() * w + (0 if d["bias"] is None else d["bias"].double().abs()))
    if d["z"] is not None:
        s = torch.nn.functional.silu(d["z"].double()).abs()
        mag = mag * s + (8 + 4 * d["z"].double().abs()) * U * want.abs()
    tol = mag + half_step(t) * (want.abs() + mag) + 1e-30
    bad = (y.double().cpu() - want).abs() > tol
    assert y.dtype == T[t] and not bad.any(), (int(bad.sum()), (y.double().cpu() - want).abs().max())
    return y


SHAPES = [(1, 1), (5, 1), (3, 2), (9, 7), (33, 16), (70, 64), (257, 64), (3, 65), (40, 128), (17, 200), (11, 256),
          (9, 512), (6, 777), (5, 1000), (8, 1024), (3, 1025), (7, 2048), (2, 4096), (2, 4097), (3, 8192), (2, 8191),
          (2, 16384), (2, 9000)]


@pytest.mark.parametrize("R,W", SHAPES)
@pytest.mark.parametrize("xt,t", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
def test_norm_fwd(gpu_lib, R, W, xt, t):
    print(f"norm_fwd R={R} W={W} {xt}->{t}", flush=True)
    for rms in (False, True):
        check_fwd(gpu_lib, make(R, W, xt, t, bias=not rms, gate=R % 2 == 1), t, rms)


def test_norm_fwd_many_rows(gpu_lib):
    """More rows than the grid holds at once, at both ends of a row's width."""
    check_fwd(gpu_lib, make(70001, 64, "bf16", "bf16", gate=True), "bf16", True)
    check_fwd(gpu_lib, make(9001, 520, "f32", "bf16"), "bf16", False)


def test_norm_fwd_no_parameters_and_large_offset(gpu_lib):
    d = make(12, 640, "f32", "f32", offset=300.0)
    check_fwd(gpu_lib, d, "f32", False)
    d["weight"] = d["bias"] = None
    check_fwd(gpu_lib, d, "f32", False)


def test_norm_strided_rows(gpu_lib):
    """Column slices of wider rows, with vector and element alignment, and a 3-D view."""
    ssd, d = gpu_lib, make(24, 96, "bf16", "bf16", gate=True)
    want = check_fwd(ssd, d, "bf16", False)
    g = up(d)
    for lead, pad in ((8, 8), (3, 2)):
        wide = torch.zeros(24, lead + 96 + pad, dtype=torch.bfloat16, device=DEV)
        wide[:, lead:lead + 96] = g["x"]
        out = torch.full_like(wide, 7.0)
        ssd.ssd_norm_fwd(wide[:, lead:lead + 96], g["weight"], bias=g["bias"], z=g["z"], y=out[:, lead:lead + 96])
        torch.testing.assert_close(out[:, lead:lead + 96].float(), want.float(), rtol=2 ** -7, atol=2 ** -12)
        assert (out[:, :lead] == 7).all() and (out[:, lead + 96:] == 7).all()
    y3 = ssd.ssd_norm_fwd(g["x"].view(4, 6, 96), g["weight"], bias=g["bias"], z=g["z"].view(4, 6, 96))
    assert torch.equal(y3.view(24, 96), want)


def test_norm_of_heads_in_wider_rows(gpu_lib):
    """Every head by itself where x, z and grad_y are column slices of wider token rows: the bits of contiguous heads."""
    ssd, (B, L, H, P) = gpu_lib, (2, 9, 4, 64)
    d = up(make(B * L * H, P, "bf16", "bf16", gate=True))
    heads = {n: d[n].view(B, L, H, P) for n in ("x", "z", "gy")}
    want = ssd.ssd_norm_fwd(d["x"], d["weight"], bias=d["bias"], z=d["z"])
    wg = ssd.ssd_norm_bwd(d["x"], d["gy"], d["weight"], bias=d["bias"], z=d["z"])
    for pad in (16, 3):
        wide = torch.zeros(3, B, L, H * P + pad, dtype=torch.bfloat16, device=DEV)
        views = {}
        for j, n in enumerate(heads):
            wide[j, ..., :H * P] = heads[n].flatten(-2)
            views[n] = wide[j, ..., :H * P].unflatten(-1, (H, P))
        y = ssd.ssd_norm_fwd(views["x"], d["weight"], bias=d["bias"], z=views["z"])
        torch.testing.assert_close(y.view(-1, P).float(), want.float(), rtol=2 ** -7, atol=2 ** -12)
        assert pad == 3 or torch.equal(y.view(-1, P), want)
        g = ssd.ssd_norm_bwd(views["x"], views["gy"], d["weight"], bias=d["bias"], z=views["z"])
        assert pad == 3 or all(torch.equal(g[n].view(wg[n].shape), wg[n]) for n in wg)
    with pytest.raises(ValueError):
        ssd.ssd_norm_fwd(views["x"].transpose(1, 2), d["weight"])


def test_norm_nan_and_inf_stay_in_their_row(gpu_lib):
    d = make(20, 256, "f32", "f32")
    d["x"][3, 5], d["x"][11, 0] = float("nan"), float("inf")
    g = up(d)
    y = gpu_lib.ssd_norm_fwd(g["x"], g["weight"], bias=g["bias"]).cpu()
    rest = [i for i in range(20) if i not in (3, 11)]
    assert torch.isnan(y[3]).all() and not torch.isfinite(y[11]).any() and torch.isfinite(y[rest]).all()


def check_bwd(ssd, d, xt, t, rms, R):
    g = up(d)
    out = ssd.ssd_norm_bwd(g["x"], g["gy"], g["weight"], bias=g["bias"], z=g["z"], rms=rms)
    leaves = {n: d[n].double().requires_grad_() for n in ("x", "weight", "bias", "z") if d[n] is not None}
    y = ref.norm(leaves["x"], leaves.get("weight"), leaves.get("bias"), leaves.get("z"), rms)
    want = dict(zip(leaves, torch.autograd.grad(y, list(leaves.values()), d["gy"].double())))
    n, rstd, off = hat_parts(d, rms)
    gy, w = d["gy"].double(), torch.ones(()) if d["weight"] is None else d["weight"].double()
    b = 0 if d["bias"] is None else d["bias"].double().abs()
    gg, rel, tol = gy, 4 * U, {}
    if d["z"] is not None:
        z = d["z"].double()
        s = torch.sigmoid(z)
        gg = gy * z * s
        rel = (16 + 4 * z.abs()) * U
        ds = (s * (1 + z * (1 - s))).abs()
        mag = gy.abs() * ((off * w.abs() + 8 * U * (n.abs() * w.abs() + b)) * ds + (n.abs() * w.abs() + b) * s * (1 + z.abs()) * rel)
        tol["z"] = mag + half_step(t) * (want["z"].abs() + mag)
    gw = (gg * w).abs()
    m1, m2 = gw.mean(-1, keepdim=True), (gw * n.abs()).mean(-1, keepdim=True)
    mag = rstd * (gw * (rel + 8 * U) + (64 * U + (rel * gw).mean(-1, keepdim=True) / (m1 + 1e-300)) * (m1 + n.abs() * m2)
                  + off * m2 + n.abs() * (gw * off).mean(-1, keepdim=True)) + 128 * U * want["x"].abs()
    tol["x"] = mag + half_step(xt) * (want["x"].abs() + mag)
    if d["weight"] is not None:
        tol["weight"] = (gg.abs() * (n.abs() * ((64 + R) * U + rel) + off)).sum(0)
    if d["bias"] is not None:
        tol["bias"] = (gg.abs() * ((64 + R) * U + rel)).sum(0)
    assert set(out) == set(want)
    for name, v in want.items():
        err = (out[name].double().cpu() - v).abs()
        assert (err <= tol[name] + 1e-30).all(), (name, err.max(), (err - tol[name]).max())
    return out


@pytest.mark.parametrize("R,W", SHAPES)
@pytest.mark.parametrize("xt,t", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
def test_norm_bwd(gpu_lib, R, W, xt, t):
    print(f"norm_bwd R={R} W={W} {xt} {t}", flush=True)
    for rms in (False, True):
        check_bwd(gpu_lib, make(R, W, xt, t, bias=not rms, gate=R % 2 == 1), xt, t, rms, R)


def test_norm_bwd_many_rows_is_deterministic(gpu_lib):
    d = make(5003, 328, "bf16", "bf16", gate=True)
    a, b = (check_bwd(gpu_lib, d, "bf16", "bf16", False, 5003) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)
    d["weight"] = d["bias"] = None
    check_bwd(gpu_lib, d, "bf16", "bf16", True, 5003)


def test_norm_bwd_against_differences(gpu_lib):
    """The gradient of sum(y * gy) against central differences of the definition in 64 bits, and of the forward call's
    own outputs in fp32 (step h: truncation h^2, rounding 2^-22 * sum |y gy| / h)."""
    d = make(3, 40, "f32", "f32", gate=True)
    g = up(d)
    out = gpu_lib.ssd_norm_bwd(g["x"], g["gy"], g["weight"], bias=g["bias"], z=g["z"])
    f = lambda e: (ref.norm(e["x"], e["weight"], e["bias"], e["z"]) * d["gy"].double()).sum()  # noqa: E731
    gen = torch.Generator().manual_seed(1)
    for name in ("x", "weight", "bias", "z"):
        way = torch.randn(d[name].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        plus, minus = (f({**d, name: d[name].double() + s * h * way}) for s in (1, -1))
        slope = (plus - minus) / (2 * h)
        got = (out[name].double().cpu() * way).sum()
        assert abs(got - slope) <= 1e-6 * (out[name].double().cpu() * way).abs().sum() + 1e-7


def test_norm_on_a_side_stream_and_captured(gpu_lib):
    """A captured forward and backward, replayed with new inputs in the same memory between eager calls."""
    ssd = gpu_lib
    d = up(make(300, 264, "bf16", "bf16", gate=True))
    ws = torch.empty(ssd.ssd_norm_bwd_workspace_size(300, 1, 264), dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call = lambda: (ssd.ssd_norm_fwd(d["x"], d["weight"], bias=d["bias"], z=d["z"]),  # noqa: E731
                        ssd.ssd_norm_bwd(d["x"], d["gy"], d["weight"], bias=d["bias"], z=d["z"], workspace=ws))
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, g = call()
    for i in range(3):
        new = up(make(300, 264, "bf16", "bf16", gate=True, seed=50 + i))
        for n in ("x", "z", "gy"):
            d[n].copy_(new[n])
        graph.replay()
        torch.cuda.synchronize()
        y1 = ssd.ssd_norm_fwd(d["x"], d["weight"], bias=d["bias"], z=d["z"])
        g1 = ssd.ssd_norm_bwd(d["x"], d["gy"], d["weight"], bias=d["bias"], z=d["z"])
        assert torch.equal(y, y1) and all(torch.equal(g[n], g1[n]) for n in g)


def test_norm_empty(gpu_lib):
    ssd = gpu_lib
    x, w = torch.zeros(0, 32, device=DEV), torch.ones(32, device=DEV)
    assert ssd.ssd_norm_fwd(x, w).shape == (0, 32)
    g = ssd.ssd_norm_bwd(x, x, w, bias=w)
    assert (g["weight"] == 0).all() and (g["bias"] == 0).all() and g["x"].shape == (0, 32)
