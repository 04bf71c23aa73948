"""GPU: ssd_delta_scan_bwd against autograd through the recurrence in 64 bits, and against differences.

Bounds, as relative L2 errors.  fp32 inputs: the forward's chain and the reverse one, each of three chained fp32 products
a chunk, and two more products behind them, of at most 128 + 64 + 64 terms each: 1024 roundings of 2^-24, 2^-14.  bf16
inputs: the fp32 outputs (dt, beta, A, dt_bias, init_state) pass at most eight split products, each off by at most 2^-15
of its terms (two operands at 2^-17, the dropped lo * lo at 2^-16): 2^-12.  q, k and v's gradients are rounded to bf16
(2^-8 at most) after products with one operand rounded (2^-8): 2^-7, with as much again for the sum of three such.
Sums over tokens (A, dt_bias) can cancel: theirs is against the sum of magnitudes of the tokens' parts."""
import pytest
import torch

from tests import delta_ref as ref
from tests.test_gpu_delta_scan import make, to_dev

pytestmark = pytest.mark.gpu

DEV = "cuda"
WIDE = {torch.float32: 2.0 ** -14, torch.bfloat16: 2.0 ** -12}
OWN = {torch.float32: 2.0 ** -14, torch.bfloat16: 2.0 ** -6}


def grads(ssd, d, opt, dims, gy, gS, *, raw=True, qk_norm=True, **kw):
    H, P, N, G = dims
    g, o = to_dev(d), to_dev(opt)
    return ssd.ssd_delta_scan_bwd(g["q"], g["k"], g["v"], g["dt"], g["A"], g["beta"], gy.to(DEV), H=H, P=P, N=N, G=G,
                                  qk_norm=qk_norm, dt_softplus=raw, beta_sigmoid=raw, dt_bias=g["dt_bias"] if raw else None,
                                  grad_final_state=None if gS is None else gS.to(DEV), **o, **kw)


def cotangents(d, opt, dims, state=True, seed=3):
    H, P, N, _ = dims
    gen = torch.Generator().manual_seed(seed)
    B, L = d["q"].shape[:2]
    gy = torch.randn(B, L, H * P, generator=gen).to(d["q"].dtype)
    return gy, torch.randn(B, H, P, N, generator=gen) if state else None


def wanted(d, opt, dims, gy, gS, *, raw=True, qk_norm=True, scale=None):
    H, P, N, G = dims
    names = [n for n in ("q", "k", "v", "dt", "A", "beta") + (("dt_bias",) if raw else ())]
    leaf = {n: d[n].double().clone().requires_grad_() for n in names}
    if opt["init_state"] is not None:
        leaf["init_state"] = opt["init_state"].double().clone().requires_grad_()
    y, S = ref.delta(*(leaf[n] for n in ("q", "k", "v", "dt", "A", "beta")), H=H, P=P, N=N, G=G, scale=scale, qk_norm=qk_norm,
                     dt_softplus=raw, beta_sigmoid=raw, dt_bias=leaf.get("dt_bias"), doc_ids=opt["doc_ids"],
                     lengths=opt["lengths"], init_state=leaf.get("init_state"))
    live = torch.ones(gy.shape[:2], dtype=torch.bool)
    if opt["lengths"] is not None:
        live = torch.arange(gy.shape[1])[None] < opt["lengths"][:, None]
    loss = (y * gy.double().masked_fill(~live[..., None], 0.0)).sum()
    if gS is not None:
        loss = loss + (S * gS.double()).sum()
    got = torch.autograd.grad(loss, list(leaf.values()), allow_unused=True)
    return {n: torch.zeros_like(leaf[n]) if g is None else g for n, g in zip(leaf, got)}, live


def check(ssd, d, opt, dims, *, state_grad=True, raw=True, **kw):
    dtype = d["q"].dtype
    if not raw:
        d = {**d, "dt": d["dt"].abs() * 0.2, "beta": torch.sigmoid(d["beta"])}
    gy, gS = cotangents(d, opt, dims, state_grad)
    out = grads(ssd, d, opt, dims, gy, gS, raw=raw, **kw)
    want, live = wanted(d, opt, dims, gy, gS, raw=raw, **kw)
    assert set(out) == set(want), (set(out), set(want))
    for name, w in want.items():
        x = out[name].double().cpu()
        assert x.shape == w.shape and torch.isfinite(x).all(), name
        if name in ("A", "dt_bias"):
            dt, _ = ref.gates(d["dt"], d["beta"], raw, d["dt_bias"] if raw else None, raw)
            part = (want["dt"].abs() / torch.sigmoid(d["dt"].double() + d["dt_bias"].double()) / d["A"].double().abs() * dt
                    if raw else want["dt"].abs() / d["A"].double().abs() * dt) if name == "A" else want["dt"].abs()
            tol = WIDE[dtype] * part.sum((0, 1))
            assert ((x - w).abs() <= tol + 1e-30).all(), (name, float(((x - w).abs() / tol).max()))
            continue
        bound = OWN[dtype] if name in ("q", "k", "v") else WIDE[dtype]
        assert (x - w).norm() <= bound * w.norm(), (name, float((x - w).norm() / w.norm()))
        if x.dim() == 3:
            assert (x[~live] == 0).all(), name
    return out


DTYPES = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("L", [1, 2, 16, 17, 63, 64, 65, 130, 200])
@pytest.mark.parametrize("dtype", DTYPES)
def test_lengths_of_a_row(gpu_lib, L, dtype):
    print(f"delta_bwd L={L} {dtype}", flush=True)
    check(gpu_lib, *make(2, L, 4, 64, 64, 2, dtype, state=True), (4, 64, 64, 2))


@pytest.mark.parametrize("B,H,P,N,G", [(1, 1, 64, 32, 1), (2, 6, 128, 32, 3), (1, 4, 128, 128, 4), (2, 4, 64, 128, 1),
                                       (3, 2, 128, 64, 2), (2, 8, 64, 64, 2)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_head_layouts(gpu_lib, B, H, P, N, G, dtype):
    print(f"delta_bwd B={B} H={H} P={P} N={N} G={G} {dtype}", flush=True)
    check(gpu_lib, *make(B, 100, H, P, N, G, dtype, packed=True), (H, P, N, G), state_grad=False)
    check(gpu_lib, *make(B, 70, H, P, N, G, dtype, state=True, docs=0.05), (H, P, N, G), raw=False, scale=0.3)


@pytest.mark.parametrize("docs", [0.02, 0.2, 1.0])
@pytest.mark.parametrize("dtype", DTYPES)
def test_documents(gpu_lib, docs, dtype):
    check(gpu_lib, *make(2, 150, 4, 64, 64, 2, dtype, docs=docs, state=True), (4, 64, 64, 2))


@pytest.mark.parametrize("dtype", DTYPES)
def test_ragged_batch(gpu_lib, dtype):
    """Rows of no, one and some tokens; NaN and Inf behind a row's length change nothing."""
    dims = (4, 64, 64, 2)
    d, opt = make(5, 130, *dims, dtype, state=True, lengths=[0, 1, 64, 65, 130])
    out = check(gpu_lib, d, opt, dims)
    gy, gS = cotangents(d, opt, dims)
    assert torch.equal(out["init_state"][0].cpu(), gS[0])
    for b, n in enumerate(opt["lengths"].tolist()):
        for t in (d["q"], d["k"], d["v"], d["dt"], d["beta"], gy):
            t[b, n:] = float("nan") if b % 2 else float("inf")
    again = grads(gpu_lib, d, opt, dims, gy, gS)
    assert all(torch.equal(out[n], again[n]) for n in out)


@pytest.mark.parametrize("dtype", DTYPES)
def test_keys_as_they_are_and_hard_gates(gpu_lib, dtype):
    dims = (2, 64, 64, 2)
    d, opt = make(2, 100, *dims, dtype, state=True)
    d["k"] = (d["k"].float() * 0.15).to(dtype)
    check(gpu_lib, d, opt, dims, qk_norm=False)
    d, opt = make(2, 130, *dims, dtype, state=True)
    d["dt"][:, 40], d["dt"][:, 100] = 1e4, 30.0
    d["beta"][:, 10:30] = -200.0
    d["v"][:, 70] = 0.0
    check(gpu_lib, d, opt, dims)


def test_every_token_its_own_document_has_no_decay_gradient(gpu_lib):
    dims = (2, 64, 64, 1)
    for dtype in DTYPES:
        d, opt = make(2, 90, *dims, dtype, docs=1.0)
        opt["doc_ids"] = torch.arange(90, dtype=torch.int32).expand(2, 90).contiguous()
        out = check(gpu_lib, d, opt, dims, state_grad=False)
        assert (out["dt"] == 0).all() and (out["A"] == 0).all()


def test_against_differences(gpu_lib):
    """The slope of the loss along a random direction of every input, by central differences in 64 bits (step 1e-4:
    truncation about 1e-8, and the direction's sum of magnitudes bounds the rounding)."""
    dims = (2, 64, 32, 1)
    H, P, N, G = dims
    d, opt = make(1, 80, *dims, torch.float32, state=True)
    gy, gS = cotangents(d, opt, dims)
    out = grads(gpu_lib, d, opt, dims, gy, gS)
    full = {**d, "init_state": opt["init_state"]}
    gen = torch.Generator().manual_seed(8)

    def loss(e):
        y, S = ref.delta(*(e[n] for n in ("q", "k", "v", "dt", "A", "beta")), H=H, P=P, N=N, G=G, qk_norm=True,
                         dt_softplus=True, beta_sigmoid=True, dt_bias=e["dt_bias"], init_state=e["init_state"])
        return (y * gy.double()).sum() + (S * gS.double()).sum()

    for name in ("q", "k", "v", "dt", "A", "beta", "dt_bias", "init_state"):
        way = torch.randn(full[name].shape, generator=gen, dtype=torch.float64)
        h = 1e-4
        slope = (loss({**full, name: full[name].double() + h * way}) - loss({**full, name: full[name].double() - h * way})) / (2 * h)
        parts = out[name].double().cpu() * way
        assert abs(parts.sum() - slope) <= 2.0 ** -14 * parts.abs().sum() + 1e-5, (name, float(parts.sum()), float(slope))


def test_repeats_bit_for_bit_and_in_a_graph(gpu_lib):
    ssd, dims = gpu_lib, (8, 64, 64, 2)
    H, P, N, G = dims
    sets = [make(2, 200, *dims, torch.bfloat16, seed=s, docs=0.02) for s in range(3)]
    cots = [cotangents(d, o, dims, False, seed=i) for i, (d, o) in enumerate(sets)]
    want = [grads(ssd, d, {**o, "doc_ids": sets[0][1]["doc_ids"]}, dims, gy, None) for (d, o), (gy, _) in zip(sets, cots)]
    g, o, gy = to_dev(sets[0][0]), to_dev(sets[0][1]), cots[0][0].to(DEV)
    ws = torch.empty(ssd.ssd_delta_scan_bwd_workspace_size(2, 200, H, P, N, G), dtype=torch.uint8, device=DEV)
    run = lambda: ssd.ssd_delta_scan_bwd(g["q"], g["k"], g["v"], g["dt"], g["A"], g["beta"], gy, H=H, P=P, N=N, G=G,  # noqa: E731
                                         qk_norm=True, dt_softplus=True, dt_bias=g["dt_bias"], beta_sigmoid=True,
                                         workspace=ws, **o)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = run()
    for i in (0, 1, 2):
        for n, v in sets[i][0].items():
            g[n].copy_(v)
        gy.copy_(cots[i][0])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(res[n], want[i][n]) for n in res)
        eager = run()
        assert all(torch.equal(eager[n], want[i][n]) for n in res)


def test_empty(gpu_lib):
    dims = (4, 64, 64, 2)
    d, opt = make(2, 0, *dims, torch.bfloat16, state=True)
    gy, gS = cotangents(d, opt, dims)
    out = grads(gpu_lib, d, opt, dims, gy, gS)
    assert (out["A"] == 0).all() and (out["dt_bias"] == 0).all() and torch.equal(out["init_state"].cpu(), gS)


def test_layer_backward(gpu_lib):
    """The layer's backward as it is used: ssd_norm_bwd, ssd_delta_scan_bwd, then the conv's (ssd_conv_bwd), in fp32,
    against autograd through the same chain in 64 bits.  Bound: the delta's, and 2^-13 more for the norm and the conv."""
    ssd, (H, P, N, G) = gpu_lib, (4, 64, 64, 2)
    B, L, dims = 2, 90, dict(H=H, P=P, N=N, G=G)
    HP, GN, Cd = H * P, G * N, H * P + 2 * G * N
    gen = torch.Generator().manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, dtr, z, w, dtb, A, beta, nw, go = (r(B, L, Cd), r(B, L, H), r(B, L, H, P), 0.5 * r(Cd, 4), r(H) - 2, -torch.exp(r(H)),
                                          r(B, L, H), 1 + 0.2 * r(P), r(B, L, H, P))
    leaf = {n: t.double().requires_grad_() for n, t in dict(x=x, dtr=dtr, z=z, w=w, A=A, beta=beta, nw=nw).items()}
    pad = torch.cat([torch.zeros(B, 3, Cd, dtype=torch.float64), leaf["x"]], 1)
    xc = torch.nn.functional.silu(sum(pad[:, k:k + L] * leaf["w"][:, k] for k in range(4)))
    y, _ = ref.delta(xc[..., HP + GN:], xc[..., HP:HP + GN], xc[..., :HP], leaf["dtr"], leaf["A"], leaf["beta"], qk_norm=True,
                     dt_softplus=True, dt_bias=dtb, beta_sigmoid=True, **dims)
    n = y.reshape(B, L, H, P)
    n = n / torch.sqrt((n * n).mean(-1, keepdim=True) + 1e-5) * leaf["nw"] * torch.nn.functional.silu(leaf["z"])
    want = dict(zip(leaf, torch.autograd.grad((n * go.double()).sum(), list(leaf.values()))))
    x, dtr, z, w, dtb, A, beta, nw, go = (t.to(DEV) for t in (x, dtr, z, w, dtb, A, beta, nw, go))
    xc, _ = ssd.ssd_conv_fwd(x, w, **dims)
    q, k, v = xc[..., HP + GN:], xc[..., HP:HP + GN], xc[..., :HP]
    kw = dict(qk_norm=True, dt_softplus=True, dt_bias=dtb, beta_sigmoid=True, **dims)
    y = ssd.ssd_delta_scan_fwd(q, k, v, dtr, A, beta, **kw)
    gn = ssd.ssd_norm_bwd(y.view(B, L, H, P), go, nw, z=z, rms=True)
    gd = ssd.ssd_delta_scan_bwd(q, k, v, dtr, A, beta, gn["x"].view(B, L, HP), **kw)
    gc = ssd.ssd_conv_bwd(x, w, torch.cat([gd["v"], gd["k"], gd["q"]], -1), **dims)
    got = dict(x=gc["raw"], dtr=gd["dt"], z=gn["z"], w=gc["w"], A=gd["A"], beta=gd["beta"], nw=gn["weight"])
    for name, g in got.items():
        err = (g.double().cpu() - want[name]).norm() / want[name].norm()
        assert err <= 2.0 ** -14 + 2.0 ** -13, (name, float(err))


@pytest.mark.parametrize("B,L,H,P,N,docs,lengths", [(1, 1500, 2, 64, 64, 0.0, None), (1, 1472, 1, 128, 128, 0.003, None),
                                                    (3, 1600, 1, 64, 32, 0.0, [0, 1600, 500])])
def test_split_sequences(gpu_lib, monkeypatch, B, L, H, P, N, docs, lengths):
    """Few heads and a long row: cut into superchunks both ways (the workspace is larger than the chunks' own).  A state
    entering one passes the chain's products twice, its own part's and the transition's: the fp32 outputs' bound doubles."""
    ssd, dims, dtype = gpu_lib, (H, P, N, 1), torch.bfloat16
    d, opt = make(B, L, *dims, dtype, state=True, docs=docs, lengths=lengths)
    units = B * H * -(-L // 64)
    chunks = units * (3 * 12288 + 9 * 256 + 4 + 8 * P * (N + 64) + 8)
    assert ssd.ssd_delta_scan_bwd_workspace_size(B, L, H, P, N, 1) > chunks + 12 * 256
    monkeypatch.setitem(WIDE, dtype, 2.0 ** -11)
    out = check(ssd, d, opt, dims)
    gy, gS = cotangents(d, opt, dims)
    again = grads(ssd, d, opt, dims, gy, gS)
    assert all(torch.equal(out[n], again[n]) for n in out)
