"""GPU: ssd_delta_scan_fwd against the recurrence in 64 bits, token by token.

Bounds, as relative L2 errors.  fp32 inputs: three chained products a chunk, on the fp32 MFMA, of at most 128 + 64 + 64
terms; 256 roundings of 2^-24 bound them even where every one of them goes the same way: 2^-16.  bf16 inputs: a split
operand (hi + lo) is off by at most 2^-17 and the dropped lo * lo product by 2^-16 of a term, and a state passes three
split products a chunk, two operands each: 3 * (2 * 2^-17 + 2^-16) = 1.5 * 2^-14 for the state.  y in bf16 rounds the
state, Att and U once (2^-8 of themselves each, at most) and itself: 4 * 2^-8.
The same bounds hold the error at every single token against the RMS of the token's own row, times 8 in place of a
maximum over the few rows that are small by cancellation."""
import pytest
import torch

from tests import delta_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
STATE = {torch.float32: 2.0 ** -16, torch.bfloat16: 1.5 * 2.0 ** -14}
Y = {torch.float32: 2.0 ** -16, torch.bfloat16: 4 * 2.0 ** -8}


def make(B, L, H, P, N, G, dtype, *, seed=0, docs=0.0, lengths=None, state=False, packed=False, decay=1.0):
    g = torch.Generator().manual_seed(1000 * seed + 7 * L + B + N + P)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    HP, GN = H * P, G * N
    silu = torch.nn.functional.silu
    if packed:
        row = silu(r(B, L, HP + 2 * GN)).to(dtype)
        v, k, q = row[..., :HP], row[..., HP:HP + GN], row[..., HP + GN:]
    else:
        v, k, q = silu(r(B, L, HP)).to(dtype), silu(r(B, L, GN)).to(dtype), silu(r(B, L, GN)).to(dtype)
    d = dict(q=q, k=k, v=v, dt=r(B, L, H), A=-decay * torch.exp(2.7 * torch.rand(H, generator=g)), beta=r(B, L, H),
             dt_bias=r(H) - 2)
    opt = dict(doc_ids=None, lengths=None, init_state=None)
    if docs:
        opt["doc_ids"] = torch.cumsum((torch.rand(B, L, generator=g) < docs).int(), 1, dtype=torch.int32)
    if lengths is not None:
        opt["lengths"] = torch.tensor(lengths, dtype=torch.int32)
    if state:
        opt["init_state"] = r(B, H, P, N)
    return d, opt


def to_dev(d):
    return {n: None if v is None else v.to(DEV) for n, v in d.items()}


def call(ssd, d, opt, dims, *, raw=True, qk_norm=True, **kw):
    H, P, N, G = dims
    g, o = to_dev(d), to_dev(opt)
    return ssd.ssd_delta_scan_fwd(g["q"], g["k"], g["v"], g["dt"], g["A"], g["beta"], H=H, P=P, N=N, G=G, qk_norm=qk_norm,
                                  dt_softplus=raw, beta_sigmoid=raw, dt_bias=g["dt_bias"] if raw else None, **o, **kw)


def compare(y, s, wy, ws, dtype, lens=None):
    y, s = y.double().cpu(), s.double().cpu()
    assert torch.isfinite(y).all() and torch.isfinite(s).all()
    es, ey = (s - ws).norm(), (y - wy).norm()
    assert es <= STATE[dtype] * ws.norm(), ("state", float(es / ws.norm()))
    assert ey <= Y[dtype] * wy.norm(), ("y", float(ey / wy.norm()))
    row = (y - wy).norm(dim=-1)
    assert (row <= 8 * Y[dtype] * wy.norm(dim=-1)).all(), ("row", (row / wy.norm(dim=-1).clamp(min=1e-300)).max())


def check(ssd, d, opt, dims, *, raw=True, qk_norm=True, **kw):
    H, P, N, G = dims
    dtype, B = d["q"].dtype, d["q"].shape[0]
    if not raw:
        d = {**d, "dt": d["dt"].abs() * 0.2, "beta": torch.sigmoid(d["beta"])}
    fs = torch.full((B, H, P, N), 3.0, device=DEV)
    y = call(ssd, d, opt, dims, raw=raw, qk_norm=qk_norm, final_state=fs, **kw)
    wy, ws = ref.delta(*(d[n] for n in ("q", "k", "v", "dt", "A", "beta")), H=H, P=P, N=N, G=G, qk_norm=qk_norm,
                       dt_softplus=raw, beta_sigmoid=raw, dt_bias=d["dt_bias"] if raw else None,
                       scale=kw.get("scale"), **opt)
    assert y.dtype == dtype
    compare(y, fs, wy, ws, dtype)
    if opt["lengths"] is not None:
        for b, n in enumerate(opt["lengths"].tolist()):
            assert (y[b, max(n, 0):] == 0).all()
    return y, fs


DTYPES = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 128, 200])
@pytest.mark.parametrize("dtype", DTYPES)
def test_lengths_of_a_row(gpu_lib, L, dtype):
    print(f"delta_scan L={L} {dtype}", flush=True)
    check(gpu_lib, *make(2, L, 4, 64, 64, 2, dtype, state=True), (4, 64, 64, 2))


@pytest.mark.parametrize("B,H,P,N,G", [(1, 1, 64, 32, 1), (2, 6, 128, 32, 3), (1, 4, 128, 128, 4), (3, 8, 64, 128, 1),
                                       (8, 2, 128, 64, 2), (4, 8, 64, 64, 2)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_head_layouts(gpu_lib, B, H, P, N, G, dtype):
    print(f"delta_scan B={B} H={H} P={P} N={N} G={G} {dtype}", flush=True)
    check(gpu_lib, *make(B, 150, H, P, N, G, dtype, packed=True), (H, P, N, G))
    check(gpu_lib, *make(B, 70, H, P, N, G, dtype, state=True, docs=0.05), (H, P, N, G), raw=False, scale=0.3)


@pytest.mark.parametrize("docs", [0.01, 0.1, 1.0])
@pytest.mark.parametrize("dtype", DTYPES)
def test_documents(gpu_lib, docs, dtype):
    check(gpu_lib, *make(3, 260, 4, 64, 64, 2, dtype, docs=docs, state=True), (4, 64, 64, 2))


@pytest.mark.parametrize("dtype", DTYPES)
def test_ragged_batch(gpu_lib, dtype):
    """Rows of 0, 1, 64, 65 and all tokens, and values outside [0, L]; padding of NaN and Inf is not read."""
    dims = (4, 64, 64, 2)
    d, opt = make(8, 190, *dims, dtype, state=True, lengths=[0, 1, 64, 65, 190, 128, -3, 1000], docs=0.02)
    y, fs = check(gpu_lib, d, opt, dims)
    assert torch.equal(fs[0].cpu(), opt["init_state"][0])
    for b, n in enumerate(opt["lengths"].clamp(0, 190).tolist()):
        for name in ("q", "k", "v", "dt", "beta"):
            d[name][b, n:] = float("nan") if b % 2 else float("inf")
    fs2 = torch.zeros_like(fs)
    y2 = call(gpu_lib, d, opt, dims, final_state=fs2)
    assert torch.equal(y, y2) and torch.equal(fs, fs2)


@pytest.mark.parametrize("dtype", DTYPES)
def test_hard_keys_and_gates(gpu_lib, dtype):
    """Equal keys with beta near 1 (the worst-conditioned inverse), no decay, total decay, beta of 0, zero rows."""
    dims = (2, 64, 64, 2)
    d, opt = make(2, 192, *dims, dtype, state=True)
    d["k"][:] = d["k"][:, :1]
    d["beta"][:] = 6.0
    d["dt"][:] = -30.0
    check(gpu_lib, d, opt, dims)
    d, opt = make(2, 130, *dims, dtype, state=True)
    d["dt"][:, 40], d["dt"][:, 100] = 1e4, float("inf")
    d["beta"][:, 10:30] = -200.0
    d["k"][:, 50], d["q"][:, 60], d["v"][:, 70] = 0.0, 0.0, 0.0
    check(gpu_lib, d, opt, dims)


def test_keys_as_they_are(gpu_lib):
    """qk_norm off: keys of length below 1 enter unscaled."""
    dims = (4, 64, 64, 2)
    for dtype in DTYPES:
        d, opt = make(2, 150, *dims, dtype)
        d["k"] = (d["k"].float() * 0.15).to(dtype)
        check(gpu_lib, d, opt, dims, qk_norm=False)


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_values(gpu_lib, dtype):
    """Values of 1e6 and 1e-6: the recurrence is linear in v and the state, and no operand's range is bounded."""
    dims = (2, 64, 32, 1)
    for f in (1e6, 1e-6):
        d, opt = make(1, 100, *dims, dtype, state=True)
        d["v"] = (d["v"].float() * f).to(dtype)
        opt["init_state"] *= f
        check(gpu_lib, d, opt, dims)


@pytest.mark.parametrize("dtype", DTYPES)
def test_state_carried_in_place_and_strided_output(gpu_lib, dtype):
    """A prefill split at 64 and 192 tokens, the state carried in place, into column slices of a wider output: the bits
    of one call, and the columns beside it untouched."""
    ssd, dims = gpu_lib, (4, 64, 64, 2)
    H, P, N, G = dims
    d, opt = make(2, 230, *dims, dtype, state=True, packed=True)
    y, fs = check(ssd, d, opt, dims)
    st = opt["init_state"].to(DEV)
    for lo, hi in ((0, 64), (64, 192), (192, 230)):
        wide = torch.full((2, hi - lo, H * P + 16), 7.0, dtype=dtype, device=DEV)
        part = {n: d[n][:, lo:hi].contiguous() if d[n].dim() == 3 else d[n] for n in d}
        g = to_dev(part)
        out = ssd.ssd_delta_scan_fwd(g["q"], g["k"], g["v"], g["dt"], g["A"], g["beta"], H=H, P=P, N=N, G=G, qk_norm=True,
                                     dt_softplus=True, beta_sigmoid=True, dt_bias=g["dt_bias"], init_state=st,
                                     final_state=st, y=wide[..., 8:8 + H * P])
        assert torch.equal(out, y[:, lo:hi]) and (wide[..., :8] == 7).all() and (wide[..., 8 + H * P:] == 7).all()
    assert torch.equal(st, fs)


def test_step_continues_the_prefill(gpu_lib):
    ssd, dims = gpu_lib, (4, 64, 128, 2)
    H, P, N, G = dims
    for dtype in DTYPES:
        d, opt = make(3, 100, *dims, dtype, state=True)
        wy, ws = ref.delta(*(d[n] for n in ("q", "k", "v", "dt", "A", "beta")), H=H, P=P, N=N, G=G, qk_norm=True,
                           dt_softplus=True, beta_sigmoid=True, dt_bias=d["dt_bias"], **opt)
        st = torch.empty(3, H, P, N, device=DEV)
        head = {n: d[n][:, :90] if d[n].dim() == 3 else d[n] for n in d}
        ys = [call(ssd, head, opt, dims, final_state=st)]
        g = to_dev(d)
        for t in range(90, 100):
            ys.append(ssd.ssd_delta_step(g["q"][:, t], g["k"][:, t], g["v"][:, t], g["dt"][:, t], g["A"], g["beta"][:, t],
                                         st, H=H, P=P, N=N, G=G, qk_norm=True, dt_softplus=True, dt_bias=g["dt_bias"],
                                         beta_sigmoid=True)[:, None])
        compare(torch.cat(ys, 1), st, wy, ws, dtype)


def test_no_state_wanted_and_empty_rows(gpu_lib):
    ssd, dims = gpu_lib, (4, 64, 64, 2)
    d, opt = make(2, 70, *dims, torch.bfloat16)
    assert torch.equal(call(ssd, d, opt, dims), check(ssd, d, opt, dims)[0])
    d, opt = make(2, 0, *dims, torch.bfloat16, state=True)
    fs = torch.zeros(2, 4, 64, 64, device=DEV)
    assert call(ssd, d, opt, dims, final_state=fs).shape == (2, 0, 256)
    assert torch.equal(fs.cpu(), opt["init_state"])
    opt["init_state"] = None
    call(ssd, d, opt, dims, final_state=fs)
    assert (fs == 0).all()


def test_two_streams_and_a_graph(gpu_lib):
    """Two calls at once on two streams with workspaces of their own, then a captured call replayed with new inputs in
    the same memory between eager calls."""
    ssd, dims = gpu_lib, (8, 64, 64, 2)
    H, P, N, G = dims
    sets = [make(2, 300, *dims, torch.bfloat16, seed=s) for s in range(4)]
    want = [call(ssd, d, o, dims) for d, o in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None] * 4
    for i, (d, o) in enumerate(sets):
        with torch.cuda.stream(streams[i % 2]):
            got[i] = call(ssd, d, o, dims)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = to_dev(sets[0][0])
    ws = torch.empty(ssd.ssd_delta_scan_workspace_size(2, 300, H, P, N, G), dtype=torch.uint8, device=DEV)
    run = lambda: ssd.ssd_delta_scan_fwd(g["q"], g["k"], g["v"], g["dt"], g["A"], g["beta"], H=H, P=P, N=N, G=G,  # noqa: E731
                                         qk_norm=True, dt_softplus=True, dt_bias=g["dt_bias"], beta_sigmoid=True, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run()
    for i in (1, 2, 3):
        for n, v in sets[i][0].items():
            g[n].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
        assert torch.equal(run(), want[i])


def test_layer_prefill_and_decode(gpu_lib):
    """The whole layer as it is used: ssd_conv_fwd over [v | k | q] and dt, the delta scan, the gated norm, then tokens
    one by one through ssd_conv_fwd at L = 1, ssd_delta_step and the norm: against the same chain in 64 bits, the conv
    output rounded to bf16 as it is stored.  Bound: y's, twice for the norm's division by a row of the same error, and
    2^-8 for the neighbouring bf16 values that the two convs may round to, for each of q, k and v."""
    ssd, (H, P, N, G) = gpu_lib, (4, 64, 64, 2)
    B, L, L1 = 2, 90, 96
    Cd = H * P + 2 * G * N
    gen = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, dtr, z = r(B, L1, Cd).bfloat16(), r(B, L1, H).bfloat16(), r(B, L1, H * P).bfloat16()
    w, dtb, A, beta, nw = 0.5 * r(Cd, 4), r(H) - 2, -torch.exp(r(H)), r(B, L1, H), 1 + 0.2 * r(P)
    pad = torch.cat([torch.zeros(B, 3, Cd, dtype=torch.float64), x.double()], 1)
    xc = torch.nn.functional.silu(sum(pad[:, k:k + L1] * w[:, k].double() for k in range(4))).bfloat16()
    v, k, q = xc[..., :H * P], xc[..., H * P:H * P + G * N], xc[..., H * P + G * N:]
    wy, _ = ref.delta(q, k, v, dtr, A, beta, H=H, P=P, N=N, G=G, qk_norm=True, dt_softplus=True, dt_bias=dtb, beta_sigmoid=True)
    want = ref.norm(wy.reshape(B, L1, H, P), nw, None, z.reshape(B, L1, H, P), True).reshape(B, L1, H * P)
    x, dtr, z, w, dtb, A, beta, nw = (t.to(DEV) for t in (x, dtr, z, w, dtb, A, beta, nw))
    dims = dict(H=H, P=P, N=N, G=G)
    cst, st = torch.zeros(B, 3, Cd, dtype=torch.bfloat16, device=DEV), torch.empty(B, H, P, N, device=DEV)
    cut = lambda c: (c[..., H * P + G * N:], c[..., H * P:H * P + G * N], c[..., :H * P])  # noqa: E731
    xc, dt = ssd.ssd_conv_fwd(x[:, :L].contiguous(), w, dt_raw=dtr[:, :L].contiguous(), dt_bias=dtb, conv_state_out=cst, **dims)
    y = ssd.ssd_delta_scan_fwd(*cut(xc), dt, A, beta[:, :L].contiguous(), qk_norm=True, beta_sigmoid=True, final_state=st, **dims)
    out = [ssd.ssd_norm_fwd(y.view(B, L, H, P), nw, z=z[:, :L].unflatten(-1, (H, P)).contiguous(), rms=True).flatten(-2)]
    for t in range(L, L1):
        xc, dt = ssd.ssd_conv_fwd(x[:, t:t + 1].contiguous(), w, dt_raw=dtr[:, t:t + 1].contiguous(), dt_bias=dtb,
                                  conv_state_in=cst, conv_state_out=cst, **dims)
        y = ssd.ssd_delta_step(*cut(xc[:, 0]), dt[:, 0], A, beta[:, t].contiguous(), st, qk_norm=True, beta_sigmoid=True, **dims)
        out.append(ssd.ssd_norm_fwd(y.view(B, H, P), nw, z=z[:, t].unflatten(-1, (H, P)), rms=True).view(B, 1, H * P))
    got = torch.cat(out, 1).double().cpu()
    bound = (2 * 4 + 3) * 2.0 ** -8
    assert (got - want).norm() <= bound * want.norm(), float((got - want).norm() / want.norm())
    assert (got[:, L:] - want[:, L:]).norm() <= bound * want[:, L:].norm()


@pytest.mark.parametrize("B,L,H,P,N,docs,lengths", [(1, 2100, 2, 64, 64, 0.0, None), (1, 2048, 1, 128, 128, 0.002, None),
                                                    (3, 2500, 1, 64, 32, 0.0, [0, 2500, 700]), (2, 2111, 2, 128, 64, 0.01, None)])
def test_split_sequences(gpu_lib, B, L, H, P, N, docs, lengths):
    """Few heads and a long row: the sequence is cut into superchunks (the workspace is larger than the chunks' own);
    with a carried state in place, documents across the cuts, and rows that end before the last superchunk."""
    ssd, dims, dtype = gpu_lib, (H, P, N, 1), torch.bfloat16
    d, opt = make(B, L, *dims, dtype, state=True, docs=docs, lengths=lengths)
    units = B * H * -(-L // 64)
    assert ssd.ssd_delta_scan_workspace_size(B, L, H, P, N, 1) > units * (10240 + 6144 + 1024 + 4) + 256
    y, fs = check(ssd, d, opt, dims)
    st = opt["init_state"].to(DEV)
    g, o = to_dev(d), to_dev({**opt, "init_state": None})
    y2 = ssd.ssd_delta_scan_fwd(g["q"], g["k"], g["v"], g["dt"], g["A"], g["beta"], H=H, P=P, N=N, G=1, qk_norm=True,
                                dt_softplus=True, beta_sigmoid=True, dt_bias=g["dt_bias"], doc_ids=o["doc_ids"],
                                lengths=o["lengths"], init_state=st, final_state=st)
    assert torch.equal(y, y2) and torch.equal(st, fs)
