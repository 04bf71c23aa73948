"""GPU: the gated linear recurrence (scan, single tokens, backward) against the definition in 64 bits.

The bounds are derived in glr_ref.py; each output in T is then rounded once, by half a step of T."""
import pytest
import torch

from tests.glr_ref import glr, masks

pytestmark = pytest.mark.gpu

DEV = "cuda"
T = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(B, L, D, t, seed=0, docs=0, lengths=False, state=False, bias=True):
    g = torch.Generator().manual_seed(seed + 7 * L + 131 * D + B)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = {n: r(B, L, D).to(T[t]) for n in ("x", "r", "i", "grad_y")}
    d["A"] = -torch.exp(torch.rand(D, generator=g) * 7.6 - 6.2)          # 0.002 .. 4
    d["r_bias"], d["i_bias"] = (0.5 * r(D), 0.5 * r(D)) if bias else (None, None)
    d["doc_ids"] = torch.cumsum((torch.rand(B, L, generator=g) < 1.0 / docs).int(), 1, dtype=torch.int32) if docs else None
    d["lengths"] = None
    if lengths:
        d["lengths"] = torch.randint(0, L + 1, (B,), generator=g, dtype=torch.int32)
        d["lengths"][0] = L
        if B > 1:
            d["lengths"][1] = 0
    d["init_state"], d["grad_final_state"] = (r(B, D), r(B, D)) if state else (None, None)
    return d


def to_dev(d):
    return {n: None if v is None else v.to(DEV) for n, v in d.items()}


FWD = ("r_bias", "i_bias", "doc_ids", "lengths", "init_state")


def fwd(ssd, g, **kw):
    B, L, D = g["x"].shape
    out = {"state": torch.full((B, D), 7.0, device=DEV), "chunk_states": torch.full((B, -(-L // 64), D), 7.0, device=DEV)}
    out["y"] = ssd.ssd_glr_scan_fwd(g["x"], g["r"], g["i"], g["A"], final_state=out["state"],
                                    chunk_states=out["chunk_states"], **{n: g[n] for n in FWD}, **kw)
    return out


def bwd(ssd, g, **kw):
    return ssd.ssd_glr_scan_bwd(g["x"], g["r"], g["i"], g["A"], g["grad_y"], grad_final_state=g["grad_final_state"],
                                **{n: g[n] for n in FWD}, **kw)


def check(got, want, tol, names=None):
    for n in names or got:
        v = want[n]
        step = torch.finfo(got[n].dtype).eps / 2
        lim = tol[n] + step * (v.abs() + tol[n]) + 1e-30
        err = (got[n].double().cpu() - v).abs()
        assert got[n].shape == v.shape and (err <= lim).all(), (n, float(err.max()), float((err / lim).max()), int((err > lim).sum()))


def reference(d, back=True):
    kw = {n: d[n] for n in FWD}
    if back:
        kw |= dict(grad_y=d["grad_y"], grad_final_state=d["grad_final_state"])
    return glr(d["x"], d["r"], d["i"], d["A"], **kw)


SHAPES = [(1, 1, 1), (2, 3, 5), (1, 8, 2), (1, 63, 128), (2, 64, 127), (3, 65, 130), (2, 127, 129), (1, 128, 64), (2, 129, 256),
          (1, 1000, 200), (2, 2100, 40), (1, 4101, 17)]


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D", SHAPES)
def test_glr_both_passes(gpu_lib, B, L, D, t):
    for k, opt in enumerate((dict(), dict(docs=1 + L // 5, lengths=True, state=True), dict(docs=2, state=True, bias=False),
                             dict(lengths=True))):
        print(f"glr B={B} L={L} D={D} {t} {opt}", flush=True)
        d = make(B, L, D, t, seed=k, **opt)
        val, tol = reference(d)
        g = to_dev(d)
        out = fwd(gpu_lib, g)
        check(out, val, tol)
        kept = bwd(gpu_lib, g, chunk_states=out["chunk_states"])
        again = bwd(gpu_lib, g)
        want = {"x", "r", "i", "A"} | ({"r_bias", "i_bias"} if opt.get("bias", True) else set()) | ({"init_state"} if opt.get("state") else set())
        assert set(kept) == set(again) == want
        check(kept, val, tol)
        assert all(torch.equal(kept[n], again[n]) for n in kept)       # the states computed again are the same
        live, _ = masks(B, L, None, d["lengths"])
        dead = (~live).expand(B, L, D).to(DEV)
        assert all((v[dead] == 0).all() for v in (out["y"], kept["x"], kept["r"], kept["i"]))


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_glr_columns_of_wider_rows(gpu_lib, t):
    """x, r, i and y as columns of wider rows, on pairs and off them; what is beside y stays."""
    for D, pad in ((130, 6), (129, 0), (64, 3), (7, 2)):
        d = make(2, 300, D, t, state=True)
        val, tol = reference(d, back=False)
        g = to_dev(d)
        wide = torch.zeros(2, 300, 3 * D + pad, dtype=T[t], device=DEV)
        for j, n in enumerate(("x", "r", "i")):
            wide[..., j * D:(j + 1) * D] = g[n]
            g[n] = wide[..., j * D:(j + 1) * D]
        out = torch.full((2, 300, D + 5), 7.0, dtype=T[t], device=DEV)
        for lead in (0, 1, 2):
            out.fill_(7.0)
            check(fwd(gpu_lib, g, y=out[..., lead:lead + D]), val, tol)
            assert (out[..., lead + D:] == 7).all() and (out[..., :lead] == 7).all()


def test_glr_nothing_behind_a_length_is_used(gpu_lib):
    d = make(4, 200, 66, "bf16", lengths=True, state=True, docs=30)
    d["lengths"] = torch.tensor([200, 0, 77, 300], dtype=torch.int32)      # the last is clamped
    live, _ = masks(4, 200, None, d["lengths"])
    clean = to_dev(d)
    for n, v in (("x", float("nan")), ("r", float("inf")), ("i", float("nan")), ("grad_y", float("inf"))):
        d[n] = torch.where(live, d[n], torch.full((), v, dtype=d[n].dtype))
    g = to_dev(d)
    a, b = fwd(gpu_lib, clean), fwd(gpu_lib, g)
    assert all(torch.equal(a[n], b[n]) for n in a)
    a, b = bwd(gpu_lib, clean), bwd(gpu_lib, g)
    assert all(torch.equal(a[n], b[n]) for n in a)
    val, tol = reference(d)
    check(b, val, tol)


def test_glr_extreme_gates(gpu_lib):
    """A of 0 (nothing forgotten, nothing taken in), decays that underflow, gates that saturate either way, a document at
    every token."""
    d = make(2, 150, 12, "f32", state=True)
    d["A"] = torch.tensor([0.0, -1e-30, -1e-6, -1e-3, -0.3499, -0.3501, -1.0, -10.0, -80.0, -1e4, -0.01, -0.05])
    d["r"][:, ::7] = 60.0
    d["r"][:, 3::7] = -60.0
    d["i"][:, 1::5] = 100.0
    d["i"][:, 2::5] = -100.0
    g = to_dev(d)
    val, tol = reference(d)
    out = fwd(gpu_lib, g)
    check(out, val, tol)
    back = bwd(gpu_lib, g)
    assert all(torch.isfinite(v).all() for v in back.values())
    # A = -1e-30 with a gate of e^-60 is below the smallest number: there the slope of sqrt(1 - a^2) is taken as 0
    fine = d["A"] != torch.tensor(-1e-30)
    for n in back:
        check({n: back[n][..., fine]}, {n: val[n][..., fine]}, {n: tol[n][..., fine]})
    assert (back["x"][..., 0] == 0).all() and (back["r"][..., 0] == 0).all()
    d["doc_ids"] = torch.arange(150, dtype=torch.int32).repeat(2, 1)
    val, tol = reference(d, back=False)
    check(fwd(gpu_lib, to_dev(d)), val, tol)


def test_glr_nan_stays_in_its_row_and_channel(gpu_lib):
    d = make(2, 500, 24, "f32")
    d["x"][1, 100, 5] = float("nan")
    y = fwd(gpu_lib, to_dev(d))["y"].cpu()
    assert torch.isnan(y[1, 100:, 5]).all() and torch.isfinite(y[1, :100, 5]).all()
    y[1, :, 5] = 0
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_glr_in_parts_and_token_by_token(gpu_lib, t):
    """A prefill in two parts with the state carried in place, then single tokens, against the whole."""
    ssd, (B, L, D) = gpu_lib, (3, 330, 72)
    d = make(B, L, D, t, state=True)
    val, tol = reference(d, back=False)
    g = to_dev(d)
    kw = dict(r_bias=g["r_bias"], i_bias=g["i_bias"])
    state, ys, at = g["init_state"].clone(), [], 0
    for n in (200, 1, 120):
        part = [g[k][:, at:at + n].contiguous() for k in ("x", "r", "i")]
        ys.append(ssd.ssd_glr_scan_fwd(*part, g["A"], init_state=state, final_state=state, **kw))
        at += n
    for k in range(at, L):
        row = [g[n][:, k] for n in ("x", "r", "i")]                # a batch row apart: strided rows
        ys.append(ssd.ssd_glr_step(*row, g["A"], state, **kw)[:, None])
    check({"y": torch.cat(ys, 1), "state": state}, val, tol)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("B,D", [(1, 1), (3, 7), (2, 8), (5, 130), (300, 64), (17, 1000)])
def test_glr_step(gpu_lib, B, D, t):
    d = make(B, 1, D, t, state=True)
    val, tol = reference(d, back=False)
    g = to_dev(d)
    for bias in (True, False):
        if not bias:
            d["r_bias"] = d["i_bias"] = g["r_bias"] = g["i_bias"] = None
            val, tol = reference(d, back=False)
        for pad in (0, 8, 1):
            row = []
            for n in ("x", "r", "i"):
                wide = torch.zeros(B, D + pad, dtype=T[t], device=DEV)
                wide[:, :D] = g[n][:, 0]
                row.append(wide[:, :D])
            state = g["init_state"].clone()
            y = gpu_lib.ssd_glr_step(*row, g["A"], state, r_bias=g["r_bias"], i_bias=g["i_bias"])
            check({"y": y[:, None], "state": state}, val, tol)


def test_glr_step_is_batch_invariant(gpu_lib):
    g = to_dev(make(9, 1, 48, "bf16", state=True))
    row, state = [g[n][:, 0].contiguous() for n in ("x", "r", "i")], g["init_state"].clone()
    y = gpu_lib.ssd_glr_step(*row, g["A"], state)
    for b in (0, 4, 8):
        one = g["init_state"][b:b + 1].clone()
        assert torch.equal(gpu_lib.ssd_glr_step(*[v[b:b + 1] for v in row], g["A"], one), y[b:b + 1]) and torch.equal(one, state[b:b + 1])


def test_glr_gradients_against_differences(gpu_lib):
    """The gradient of sum(y gy) + sum(state gs) along random directions against central differences of the definition."""
    d = make(2, 90, 10, "f32", docs=20, lengths=True, state=True)
    d["lengths"][1] = 60
    back = bwd(gpu_lib, to_dev(d))
    gen = torch.Generator().manual_seed(5)

    def f(e):
        val, _ = glr(e["x"], e["r"], e["i"], e["A"], **{n: e[n] for n in FWD})
        return (val["y"] * d["grad_y"].double()).sum() + (val["state"] * d["grad_final_state"].double()).sum()

    for name in ("x", "r", "i", "A", "r_bias", "i_bias", "init_state"):
        way = torch.randn(d[name].shape, generator=gen, dtype=torch.float64)
        if name == "A":
            way = way * d["A"].double().abs()              # a direction that keeps A negative
        h = 1e-5
        plus, minus = (f({**d, name: d[name].double() + k * h * way}) for k in (1, -1))
        got = back[name].double().cpu() * way
        # truncation of order h^2 and the kernels' errors, some 1e-6 of the terms' magnitudes
        assert abs(got.sum() - (plus - minus) / (2 * h)) <= 2e-5 * got.abs().sum() + 1e-7, name


def test_glr_runs_alike(gpu_lib):
    """The same bits from call to call, with poisoned workspaces, of rows of many tiles."""
    ssd = gpu_lib
    g = to_dev(make(2, 9000, 200, "bf16", docs=700, state=True))
    first = None
    for fill in (0, 255, 127):
        ws = torch.full((ssd.ssd_glr_scan_workspace_size(2, 9000, 200),), fill, dtype=torch.uint8, device=DEV)
        wb = torch.full((ssd.ssd_glr_scan_bwd_workspace_size(2, 9000, 200),), fill, dtype=torch.uint8, device=DEV)
        out = fwd(ssd, g, workspace=ws)
        out |= {"d" + n: v for n, v in bwd(ssd, g, workspace=wb, chunk_states=out["chunk_states"] if fill else None).items()}
        first = first or out
        assert all(torch.equal(out[n], first[n]) for n in out)


def test_glr_long_rows(gpu_lib):
    """Thousands of tokens that a slow channel remembers, in many tiles: against the definition on the GPU in 64 bits."""
    B, L, D = 1, 40000, 130
    d = make(B, L, D, "f32", state=True, docs=9000)
    d["A"][:64] = -0.002
    g = to_dev(d)
    out = fwd(gpu_lib, g)
    s = torch.sigmoid(g["r"].double() + g["r_bias"].double())
    a = torch.exp(s * g["A"].double())
    b = torch.sqrt(-torch.expm1(2 * s * g["A"].double())) * torch.sigmoid(g["i"].double() + g["i_bias"].double()) * g["x"].double()
    fresh = masks(B, L, d["doc_ids"])[1].to(DEV)
    a = torch.where(fresh, 0.0, a)
    h, hs = g["init_state"].double(), []
    for t in range(L):
        h = a[:, t] * h + b[:, t]
        hs.append(h)
    hs = torch.stack(hs, 1)
    # a decay is off by 2 U + n (12 + 2|v|) U and the state remembers 1 / (1 - a) of them: relative to its magnitude,
    # (14 + 2|v|) U times at most a few; 1e-4 would be one step the same way at each token of the slowest channels
    assert float((out["y"].double() - hs).norm() / hs.norm()) < 2e-6
    assert float((out["state"].double() - hs[:, -1]).norm() / hs[:, -1].norm()) < 4e-6


def test_glr_rows_past_4g_bytes(gpu_lib):
    """Rows whose elements lie past 2^32 bytes and past 2^31 elements."""
    L, D, stride = 70000, 6, 32770
    base = torch.empty(L * stride, dtype=torch.bfloat16, device=DEV)
    wide = base.view(1, L, stride)
    d = to_dev(make(1, L, D, "bf16", docs=5000))
    want = gpu_lib.ssd_glr_scan_fwd(d["x"], d["r"], d["i"], d["A"], doc_ids=d["doc_ids"])
    view = {}
    for j, n in enumerate(("x", "r", "i")):
        view[n] = wide[..., j * D:(j + 1) * D]
        view[n].copy_(d[n])
    y = wide[..., 20:20 + D]
    gpu_lib.ssd_glr_scan_fwd(view["x"], view["r"], view["i"], d["A"], doc_ids=d["doc_ids"], y=y)
    assert torch.equal(y.contiguous(), want)


def test_glr_on_streams_and_captured(gpu_lib):
    """Given a stream; two calls at once on two streams; captured and replayed with new inputs between eager calls."""
    ssd = gpu_lib
    sets = [to_dev(make(2, 5000, 300, "bf16", seed=s, state=True, docs=600)) for s in range(3)]
    want = [(fwd(ssd, g), bwd(ssd, g)) for g in sets]
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        got = [(fwd(ssd, g, stream=s), bwd(ssd, g, stream=s)) for g, s in zip(sets, (one, two, one))]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u[n], v[n]) for u, v in zip(a, b) for n in v)
    g = {n: None if v is None else v.clone() for n, v in sets[0].items()}
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        fwd(ssd, g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fwd(ssd, g)
        back = bwd(ssd, g, chunk_states=out["chunk_states"])
    for k in (1, 2, 0, 1):
        for n, v in sets[k].items():
            if v is not None:
                g[n].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], want[k][0][n]) for n in out) and all(torch.equal(back[n], want[k][1][n]) for n in back)
        eager = fwd(ssd, sets[k])
        assert torch.equal(eager["y"], want[k][0]["y"])


def test_glr_empty(gpu_lib):
    ssd = gpu_lib
    A = -torch.ones(6, device=DEV)
    x = torch.zeros(3, 0, 6, device=DEV)
    h0, hf = torch.randn(3, 6, device=DEV), torch.full((3, 6), 7.0, device=DEV)
    assert ssd.ssd_glr_scan_fwd(x, x, x, A, init_state=h0, final_state=hf).shape == (3, 0, 6) and torch.equal(hf, h0)
    ssd.ssd_glr_scan_fwd(x, x, x, A, final_state=hf)
    assert (hf == 0).all()
    g = ssd.ssd_glr_scan_bwd(x, x, x, A, x, init_state=h0, grad_final_state=h0, r_bias=A, i_bias=A)
    assert torch.equal(g["init_state"], h0) and all((g[n] == 0).all() for n in ("A", "r_bias", "i_bias"))
    e = torch.zeros(0, 9, 6, device=DEV)
    assert ssd.ssd_glr_scan_fwd(e, e, e, A).shape == (0, 9, 6)
    g = ssd.ssd_glr_scan_bwd(e, e, e, A, e, r_bias=A)
    assert (g["A"] == 0).all() and (g["r_bias"] == 0).all() and g["x"].shape == (0, 9, 6)
    assert ssd.ssd_glr_step(e[:, 0], e[:, 0], e[:, 0], A, torch.zeros(0, 6, device=DEV)).shape == (0, 6)


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_glr_documents_keep_nan_to_themselves(gpu_lib, t):
    """NaN and infinities in a document reach no other: the state of later ones (within a stretch, a tile and across
    tiles), and the gradients of earlier ones.  Behind a row's length gradients are 0 whatever the row holds."""
    ssd, (B, L, D) = gpu_lib, (2, 2500, 34)
    d = make(B, L, D, t, state=True)
    cuts = [0, 3, 70, 400, 1500, 2400]
    ids = torch.zeros(L, dtype=torch.int32)
    for c in cuts:
        ids[c:] += 1
    d["doc_ids"], d["lengths"] = ids.repeat(B, 1), torch.tensor([L, 2450], dtype=torch.int32)
    g = to_dev(d)
    clean, cleanb = fwd(ssd, g), bwd(ssd, g)
    for lo, hi in zip(cuts, cuts[1:] + [L]):
        e = {n: None if v is None else v.clone() for n, v in g.items()}
        e["x"][:, lo, ::2], e["r"][:, lo, 1::2] = float("inf"), float("nan")
        if lo == 0:
            e["init_state"].fill_(float("nan"))
        y = fwd(ssd, e)["y"]
        out = [k for k in range(L) if not lo <= k < hi]
        assert torch.equal(y[:, out], clean["y"][:, out]) and not torch.isfinite(y[0, hi - 1]).any()
        e = {n: None if v is None else v.clone() for n, v in g.items()}
        e["grad_y"][:, hi - 1] = float("nan")
        if hi == L:
            e["grad_final_state"].fill_(float("inf"))
        back = bwd(ssd, e)
        for n in ("x", "r", "i"):
            assert torch.equal(back[n][:, out], cleanb[n][:, out]) and (back[n][1, 2450:] == 0).all()
    e = {n: None if v is None else v.clone() for n, v in g.items()}
    e["x"][1, 2449] = float("inf")
    assert all((bwd(ssd, e)[n][1, 2450:] == 0).all() for n in ("x", "r", "i"))
