"""GPU: ssd_add_norm_fwd and ssd_add_norm_bwd against the definition in 64 bits.

Bounds.  The sum is one fp32 addition and one rounding: compared exactly.  The norm of the stored sum is ssd_norm_fwd's:
a statistic is off by at most 42 * 2^-24 of its sum of magnitudes, and 64 * 2^-24 covers one pass (test_gpu_norm.py).  A
block's scale inherits the error of its largest |y|, and two roundings.  q is the e4m3 number nearest to y / scale: half a
step is 2^-4 of it, or 2^-10 scale below the smallest normal number."""
import pytest
import torch

from tests import delta_ref as ref
from tests.test_gpu_norm import SHAPES, U, half_step

pytestmark = pytest.mark.gpu

DEV = "cuda"
T = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(R, W, xt, rt, t, residual=True, bias=True, gate=False, seed=0):
    g = torch.Generator().manual_seed(seed + 31 * W + R)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(x=(r(R, W) * 2 + 0.5).to(T[xt]), residual=r(R, W).to(T[rt]) if residual else None, weight=1 + 0.3 * r(W),
             bias=0.3 * r(W) if bias else None, z=r(R, W).to(T[t]) if gate else None, gy=r(R, W).to(T[t]),
             gs=r(R, W).to(T[rt]))
    d["sum"] = (d["x"].float() + d["residual"].float()).to(T[rt]) if residual else d["x"]
    return d


def up(d):
    return {n: None if v is None else v.to(DEV) for n, v in d.items()}


def hat_parts(s, rms):
    s = s.double()
    c = s if rms else s - s.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5)
    n = c * rstd
    return n, rstd, 64 * U * (2 * n.abs() + (0.0 if rms else 1.0) * s.abs().mean(-1, keepdim=True) * rstd)


def blocks(y):
    """[R, W] -> [R, blocks, 128], filled up with zeros."""
    R, W = y.shape
    pad = torch.zeros(R, -(-W // 128) * 128, dtype=y.dtype, device=y.device)
    pad[:, :W] = y
    return pad.view(R, -1, 128)


def run(ssd, g, t, rms, **kw):
    return ssd.ssd_add_norm_fwd(g["x"], g["residual"], g["weight"], bias=g["bias"], z=g["z"], rms=rms, out_dtype=T[t], **kw)


def check_fwd(ssd, d, t, rms):
    g = up(d)
    out = run(ssd, g, t, rms, want_q=True)
    R, W = d["x"].shape
    assert set(out) == {"y", "q", "scale"} | ({"sum"} if d["residual"] is not None else set())
    if d["residual"] is not None:
        assert out["sum"].dtype == d["sum"].dtype and torch.equal(out["sum"].cpu(), d["sum"])
    want = ref.norm(d["sum"], d["weight"], d["bias"], d["z"], rms)
    n, _, off = hat_parts(d["sum"], rms)
    w = torch.ones(()) if d["weight"] is None else d["weight"].double().abs()
    mag = off * w + 4 * U * (n.abs() * w + (0 if d["bias"] is None else d["bias"].double().abs()))
    if d["z"] is not None:
        s = torch.nn.functional.silu(d["z"].double()).abs()
        mag = mag * s + (8 + 4 * d["z"].double().abs()) * U * want.abs()
    tol = mag + half_step(t) * (want.abs() + mag) + 1e-30
    err = (out["y"].double().cpu() - want).abs()
    assert out["y"].dtype == T[t] and (err <= tol).all(), (int((err > tol).sum()), err.max())
    top, slack = blocks(want).abs().amax(-1), blocks(mag).amax(-1)
    scale = out["scale"].double().cpu()
    near = (scale - top / 448).abs() <= slack / 448 + 4 * U * top / 448 + 2.0 ** -100
    assert (near | ((scale == 1) & (top <= slack))).all()      # a maximum within its error of 0 may be 0, whose scale is 1
    wide = scale.repeat_interleave(128, 1)[:, :W]
    q = out["q"].double().cpu()
    lim = mag * (1 + 2.0 ** -4) + (2.0 ** -4 + 8 * U) * want.abs() + 2.0 ** -10 * wide
    assert ((q * wide - want).abs() <= lim).all(), float(((q * wide - want).abs() / lim).max())
    # one output alone is what it is beside the other, and a y in fp32 quantises to q exactly
    alone = run(ssd, g, t, rms, want_y=False, want_q=True)
    assert "y" not in alone and torch.equal(alone["q"].view(torch.uint8), out["q"].view(torch.uint8)) and torch.equal(alone["scale"], out["scale"])
    alone = run(ssd, g, t, rms)
    assert "q" not in alone and torch.equal(alone["y"], out["y"])
    if t == "f32":
        inv = (1.0 / out["scale"]).repeat_interleave(128, 1)[:, :W]
        assert torch.equal((out["y"] * inv).clamp(-448, 448).to(torch.float8_e4m3fn).float(), out["q"].float())
    return out


@pytest.mark.parametrize("R,W", SHAPES)
@pytest.mark.parametrize("xt,rt,t", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("bf16", "f32", "bf16"), ("f32", "bf16", "f32")])
def test_add_norm_fwd(gpu_lib, R, W, xt, rt, t):
    print(f"add_norm_fwd R={R} W={W} {xt} + {rt} -> {t}", flush=True)
    for rms in (False, True):
        check_fwd(gpu_lib, make(R, W, xt, rt, t, bias=not rms, gate=R % 2 == 1), t, rms)
        check_fwd(gpu_lib, make(R, W, xt, rt, t, residual=False, bias=rms, gate=R % 2 == 0), t, rms)


def test_add_norm_many_rows(gpu_lib):
    check_fwd(gpu_lib, make(70001, 64, "bf16", "bf16", "bf16", gate=True), "bf16", True)
    check_fwd(gpu_lib, make(9001, 520, "f32", "f32", "bf16"), "bf16", False)
    check_fwd(gpu_lib, make(9001, 131, "bf16", "f32", "f32"), "f32", True)


def test_add_norm_in_place_and_strided(gpu_lib):
    """The sum in place of the residual or of x; columns of wider rows, with vector and element alignment."""
    ssd = gpu_lib
    for W, lead, pad in ((96, 8, 8), (96, 3, 2), (200, 16, 24), (77, 1, 0)):
        d = make(24, W, "bf16", "bf16", "bf16", gate=True)
        want = check_fwd(ssd, d, "bf16", True)
        g = up(d)
        res = g["residual"].clone()
        got = run(ssd, {**g, "residual": res}, "bf16", True, sum=res, want_q=True)
        assert got["sum"] is res and torch.equal(res, want["sum"]) and torch.equal(got["y"], want["y"])
        x = g["x"].clone()
        got = run(ssd, {**g, "x": x}, "bf16", True, sum=x, want_q=True)
        assert torch.equal(x, want["sum"]) and torch.equal(got["y"], want["y"])
        room = {}
        for n in ("x", "residual", "z"):
            wide = torch.zeros(24, lead + W + pad, dtype=torch.bfloat16, device=DEV)
            wide[:, lead:lead + W] = g[n]
            room[n] = wide[:, lead:lead + W]
        y = torch.full((24, lead + W + pad), 7.0, dtype=torch.bfloat16, device=DEV)
        q = torch.full((24, lead + W + pad), 7.0, device=DEV).to(torch.float8_e4m3fn)
        scale = torch.full((24, 5), 7.0, device=DEV)
        nb = -(-W // 128)
        got = run(ssd, {**g, **room}, "bf16", True, sum=room["residual"], y=y[:, lead:lead + W], q=q[:, lead:lead + W],
                  q_scale=scale[:, 1:1 + nb])
        torch.testing.assert_close(got["y"].float(), want["y"].float(), rtol=2 ** -7, atol=2 ** -12)
        torch.testing.assert_close(got["scale"], want["scale"], rtol=1e-5, atol=0)
        torch.testing.assert_close(got["q"].float(), want["q"].float(), rtol=2 ** -3, atol=2 ** -9)
        for t, n in ((y, W), (q.float(), W)):
            assert (t[:, :lead] == 7).all() and (t[:, lead + n:] == 7).all()
        assert (scale[:, 0] == 7).all() and (scale[:, 1 + nb:] == 7).all()


@pytest.mark.parametrize("W", [256, 250])
def test_add_norm_blocks_of_zeros_nan_and_infinities(gpu_lib, W):
    """eps under the root of rows that are all zero; a weight of 0, infinity or NaN makes a block's values."""
    d = make(6, W, "f32", "f32", "f32", residual=False, bias=False)
    d["x"][2] = 0.0
    d["x"][3, 7] = float("nan")
    d["x"][5] *= 1e-25                                # a row far below eps: y as small as 1e-23
    d["weight"][128:] = 0.0
    out = run(gpu_lib, up(d), "f32", True, want_q=True)
    q, scale = out["q"].float().cpu(), out["scale"].cpu()
    rows = [0, 1, 4, 5]
    assert torch.isfinite(q[rows]).all() and torch.isfinite(scale).all() and (scale > 0).all()
    assert (scale[rows, 1] == 1).all() and (q[rows, 128:] == 0).all()
    assert (scale[2] == 1).all() and (q[2] == 0).all()
    assert torch.isnan(q[3]).all() and (scale[3] == 1).all()
    assert ((q[5] * scale[5].repeat_interleave(128)[:W] - out["y"].cpu()[5]).abs() <= (2 ** -4 + 8 * U) * out["y"].cpu()[5].abs() + 2.0 ** -10 * scale[5, 0]).all()
    d = make(3, W, "f32", "f32", "f32", residual=False, bias=False)
    d["weight"][5], d["weight"][6] = float("inf"), -float("inf")
    d["weight"][9] = float("nan")
    out = run(gpu_lib, up(d), "f32", True, want_q=True)
    q, scale = out["q"].float().cpu(), out["scale"].cpu()
    assert torch.equal(q[:, 5].sign(), d["x"][:, 5].sign()) and (q[:, 5:7].abs() == 448).all() and torch.isnan(q[:, 9]).all()
    keep = [c for c in range(W) if c != 9]
    assert torch.isfinite(q[:, keep]).all() and torch.isfinite(scale).all()
    assert (q[:, 128:].abs().amax(1) == 448).all()


def check_bwd(ssd, d, rt, t, rms, past=True):
    g = up(d)
    out = ssd.ssd_add_norm_bwd(g["sum"], g["gy"], g["gs"] if past else None, g["weight"], bias=g["bias"], z=g["z"], rms=rms)
    R = d["sum"].shape[0]
    leaves = {n: d[n].double().requires_grad_() for n in ("sum", "weight", "bias", "z") if d[n] is not None}
    y = ref.norm(leaves["sum"], leaves.get("weight"), leaves.get("bias"), leaves.get("z"), rms)
    want = dict(zip(leaves, torch.autograd.grad(y, list(leaves.values()), d["gy"].double())))
    n, rstd, off = hat_parts(d["sum"], rms)
    gy, w = d["gy"].double(), torch.ones(()) if d["weight"] is None else d["weight"].double()
    b = 0 if d["bias"] is None else d["bias"].double().abs()
    gg, rel, tol = gy, 4 * U, {}
    if d["z"] is not None:
        z = d["z"].double()
        s = torch.sigmoid(z)
        gg, rel = gy * z * s, (16 + 4 * z.abs()) * U
        ds = (s * (1 + z * (1 - s))).abs()
        mag = gy.abs() * ((off * w.abs() + 8 * U * (n.abs() * w.abs() + b)) * ds + (n.abs() * w.abs() + b) * s * (1 + z.abs()) * rel)
        tol["z"] = mag + half_step(t) * (want["z"].abs() + mag)
    gw = (gg * w).abs()
    m1, m2 = gw.mean(-1, keepdim=True), (gw * n.abs()).mean(-1, keepdim=True)
    mag = rstd * (gw * (rel + 8 * U) + (64 * U + (rel * gw).mean(-1, keepdim=True) / (m1 + 1e-300)) * (m1 + n.abs() * m2)
                  + off * m2 + n.abs() * (gw * off).mean(-1, keepdim=True)) + 128 * U * want["sum"].abs()
    if past:
        want["sum"] = want["sum"] + d["gs"].double()
        mag = mag + 2 * U * want["sum"].abs()
    tol["sum"] = mag + half_step(rt) * (want["sum"].abs() + mag)
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
@pytest.mark.parametrize("rt,t", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
def test_add_norm_bwd(gpu_lib, R, W, rt, t):
    print(f"add_norm_bwd R={R} W={W} {rt} {t}", flush=True)
    for rms in (False, True):
        d = make(R, W, "f32", rt, t, bias=not rms, gate=R % 2 == 1)
        check_bwd(gpu_lib, d, rt, t, rms)
        check_bwd(gpu_lib, d, rt, t, rms, past=False)


def test_add_norm_bwd_many_rows_in_place(gpu_lib):
    """Deterministic; dsum in place of grad_sum through the C ABI's own arguments."""
    ssd = gpu_lib
    d = make(5003, 328, "bf16", "bf16", "bf16", gate=True)
    a, b = (check_bwd(ssd, d, "bf16", "bf16", False) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)
    d["weight"] = d["bias"] = d["z"] = None
    want = check_bwd(ssd, d, "bf16", "bf16", True)["sum"]
    g = up(d)
    st = ssd.load().ssd_add_norm_bwd(5003, 328, 1, 1, 1, 1e-5, g["sum"].data_ptr(), 328, None, None, None, 0, g["gy"].data_ptr(), 328,
                                     g["gs"].data_ptr(), 328, g["gs"].data_ptr(), 328, None, None, None, 0, None, 0,
                                     torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(g["gs"], want)


def test_add_norm_gradients_against_differences(gpu_lib):
    """The gradient of sum(y gy) + sum(s gs) against central differences of the definition."""
    d = make(3, 40, "f32", "f32", "f32", gate=True)
    g = up(d)
    out = gpu_lib.ssd_add_norm_bwd(g["sum"], g["gy"], g["gs"], g["weight"], bias=g["bias"], z=g["z"])
    f = lambda e: (ref.norm(e["sum"], e["weight"], e["bias"], e["z"]) * d["gy"].double()).sum() + (e["sum"].double() * d["gs"].double()).sum()  # noqa: E731
    gen = torch.Generator().manual_seed(1)
    for name in ("sum", "weight", "bias", "z"):
        way = torch.randn(d[name].shape, generator=gen, dtype=torch.float64)
        plus, minus = (f({**d, name: d[name].double() + s * 1e-5 * way}) for s in (1, -1))
        got = (out[name].double().cpu() * way)
        assert abs(got.sum() - (plus - minus) / 2e-5) <= 1e-6 * got.abs().sum() + 1e-7


def test_add_norm_on_a_stream_captured_and_empty(gpu_lib):
    ssd = gpu_lib
    sets = [up(make(300, 1000, "bf16", "f32", "bf16", seed=s)) for s in range(3)]

    def both(g, **kw):
        out = run(ssd, g, "bf16", True, want_q=True, **kw)
        return out | {"d" + n: v for n, v in ssd.ssd_add_norm_bwd(out["sum"], g["gy"], g["gs"], g["weight"], bias=g["bias"], rms=True, **kw).items()}

    same = lambda a, b: all(torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)) for n in b)  # noqa: E731
    want = [both(g) for g in sets]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = both(sets[0], stream=s)
    torch.cuda.synchronize()
    assert same(got, want[0])
    g = {n: None if v is None else v.clone() for n, v in sets[0].items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(g)
    for k in (1, 2, 0):
        for n, v in sets[k].items():
            if v is not None:
                g[n].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, want[k]) and same(both(sets[k]), want[k])
    e = torch.zeros(0, 48, device=DEV)
    out = ssd.ssd_add_norm_fwd(e, e, want_q=True)
    assert out["q"].shape == (0, 48) and out["scale"].shape == (0, 1) and out["sum"].shape == (0, 48)
    back = ssd.ssd_add_norm_bwd(e, e, e, torch.ones(48, device=DEV), bias=torch.ones(48, device=DEV))
    assert (back["weight"] == 0).all() and (back["bias"] == 0).all()


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_add_norm_ends_of_rows(gpu_lib, t):
    """Rows that end at every place of a vector and start at every alignment: nothing past a row's end is read (it is NaN) or
    written, forward and backward."""
    ssd, e4 = gpu_lib, torch.float8_e4m3fn
    for W in list(range(1, 20)) + [63, 65, 127, 129, 255, 257, 1023, 1031, 2079]:
        for lead, pad in ((0, 1), (1, 2), (3, 4), (8, 8)):
            d = make(9, W, t, t, t, gate=True)
            g = up(d)

            def wide(v, fill=float("nan")):
                out = torch.full((9, lead + W + pad), fill, dtype=v.dtype, device=DEV)
                out[:, lead:lead + W] = v
                return out[:, lead:lead + W], out

            def clean(out):
                edge = out.float()
                return bool((edge[:, :lead] == 7).all() and (edge[:, lead + W:] == 7).all())
            ins = {n: wide(g[n])[0] for n in ("x", "residual", "z", "gy", "gs")}
            outs = {n: wide(torch.zeros(9, W, dtype=T[t], device=DEV), 7.0) for n in ("sum", "y")}
            outs["q"] = wide(torch.zeros(9, W, device=DEV), 7.0)[1].to(e4)
            q = outs["q"][:, lead:lead + W]
            got = ssd.ssd_add_norm_fwd(ins["x"], ins["residual"], g["weight"], bias=g["bias"], z=ins["z"], rms=False, sum=outs["sum"][0],
                                       y=outs["y"][0], q=q)
            want = run(ssd, g, t, False, want_q=True)
            for n in ("sum", "y", "scale"):
                assert torch.equal(got[n], want[n]), (W, lead, n)
            assert torch.equal(q.contiguous().view(torch.uint8), want["q"].view(torch.uint8)) and clean(outs["q"])
            assert clean(outs["sum"][1]) and clean(outs["y"][1])
            for gs in (None, "gs"):
                a = ssd.ssd_add_norm_bwd(outs["sum"][0], ins["gy"], gs and ins[gs], g["weight"], bias=g["bias"], z=ins["z"])
                b = ssd.ssd_add_norm_bwd(want["sum"], g["gy"], gs and g[gs], g["weight"], bias=g["bias"], z=g["z"])
                assert set(a) == {"sum", "z", "weight", "bias"} and all(torch.equal(a[n], b[n]) for n in a), (W, lead, gs)
