"""Cases for measuring the gated delta rule (prefill, single tokens, backward pass) and the row norm (both passes).

The gated delta rule keeps, for each sequence and head, a state S [N, P] and reads one token after the other:

    S <- a S,  u = beta (v - S^T k),  S <- S + k u^T,  y = scale S^T q,      a = exp(dt A)

The row norm maps a row x of W columns to (x - mean) * rstd * weight + bias (or x * rstd * weight, the mean
square in place of the variance), times silu(z) where there is a gate.

With `own` false, run() computes them in elementary torch operations, in 32 bits (decays in 64); with `own`
true it calls this repository's package.
"""
import math

import torch

own = False

QK_EPS = 1e-6      # under the root of the q and k normalisation
CHUNK = 64         # tokens of one block of the plain form


def listed():
    return [
        # a ragged batch of short prompts, one of them empty: what a server collects in one go; latency counts
        dict(name="delta_fwd_f32_ragged", op="delta_fwd", dtype="f32", B=3, L=77, H=8, P=64, N=64, G=2, docs=0,
             lengths=True, state=True, packed=False, raw=True),
        # packed documents of a training batch at the repository's 32-head, 64-channel, state-64 mixer shape
        dict(name="delta_fwd_bf16_docs", op="delta_fwd", dtype="bf16", B=5, L=8192, H=32, P=64, N=64, G=8, docs=1024,
             lengths=False, state=False, packed=False, raw=True),
        # the large layer: many heads, state 128, a carried state, q k v as columns of one conv output
        dict(name="delta_fwd_bf16_large", op="delta_fwd", dtype="bf16", B=4, L=4096, H=128, P=64, N=128, G=8, docs=0,
             lengths=False, state=True, packed=True, raw=True),
        # one long prompt: few rows, a long axis
        dict(name="delta_fwd_bf16_long", op="delta_fwd", dtype="bf16", B=1, L=32768, H=16, P=128, N=128, G=16, docs=0,
             lengths=False, state=False, packed=True, raw=True),
        # one sequence's next token: latency alone
        dict(name="delta_step_bf16_one", op="delta_step", dtype="bf16", B=1, H=32, P=64, N=64, G=8, packed=True,
             raw=True),
        # the decode batch: 256 sequences, 64 heads, state 128; the state's bytes are the work
        dict(name="delta_step_f32_batch", op="delta_step", dtype="f32", B=256, H=64, P=64, N=128, G=1, packed=False,
             raw=False),
        # a small training step in 32 bits with odd lengths and a carried state, its gradient among the outputs
        dict(name="delta_bwd_f32_small", op="delta_bwd", dtype="f32", B=2, L=150, H=4, P=64, N=32, G=2, docs=50,
             lengths=True, state=True, packed=False, raw=True),
        # a training step at the 32-head mixer shape with packed documents
        dict(name="delta_bwd_bf16_docs", op="delta_bwd", dtype="bf16", B=2, L=8192, H=32, P=64, N=64, G=8, docs=1024,
             lengths=False, state=False, packed=True, raw=True),
        # the norm of the mixer's fp32 output on its way to a bf16 projection: rows of H*P columns
        dict(name="norm_fwd_scan_y", op="norm_fwd", xdtype="f32", dtype="bf16", R=40960, W=2048, rms=False, bias=True,
             gate=False),
        # a gated norm of every head by itself: very many short rows
        dict(name="norm_fwd_heads_gated", op="norm_fwd", xdtype="bf16", dtype="bf16", R=1310720, W=64, rms=True,
             bias=False, gate=True),
        # odd sizes: rows that no vector load divides
        dict(name="norm_bwd_f32_odd", op="norm_bwd", xdtype="f32", dtype="f32", R=333, W=1001, rms=False, bias=True,
             gate=False),
        # the gated norm's training step over a whole batch of rows
        dict(name="norm_bwd_bf16_gated", op="norm_bwd", xdtype="bf16", dtype="bf16", R=40960, W=2048, rms=False,
             bias=True, gate=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_fwd", "delta_step", "delta_bwd", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["f32", "bf16", "bf16"])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op.startswith("norm"):
        W = _log_int(rng, 16, 12000)
        R = _log_int(rng, 1, max(2, min(600000, 60_000_000 // W)))
        if flag() or W > 8000:
            W = -(-W // 8) * 8
        return dict(op=op, xdtype=rng.choice([dtype, "f32"]), dtype=dtype, R=R, W=W, rms=flag(), bias=flag(), gate=flag())
    G = rng.choice([1, 2, 4, 8])
    c = dict(op=op, dtype=dtype, H=G * rng.choice([1, 2, 3, 4]), P=rng.choice([64, 128]), N=rng.choice([32, 64, 128]), G=G,
             packed=flag(), raw=flag())
    if op == "delta_step":
        c["B"] = _log_int(rng, 1, 300)
        return c
    c["B"] = rng.randint(1, 8)
    cap = (8e9 if op == "delta_fwd" else 1.5e9) / (c["B"] * c["H"] * c["P"] * c["N"])
    c["L"] = _log_int(rng, 1, max(2, min(16384 if op == "delta_fwd" else 4096, int(cap))))
    c["docs"] = rng.choice([0, 0, 1 + c["L"] // 7])
    c["lengths"] = rng.random() < 0.3
    c["state"] = flag()
    return c


def _dt(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 17)
    randn = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=gen, device=dev)  # noqa: E731
    c, st = case, {"case": case}
    T = _dt(c["dtype"])
    if c["op"].startswith("norm"):
        R, W = c["R"], c["W"]
        st["x"] = (randn(R, W) * 1.5 + 0.25).to(_dt(c["xdtype"]))
        st["weight"] = 1.0 + 0.2 * randn(W)
        st["bias"] = 0.2 * randn(W) if c["bias"] else None
        st["z"] = randn(R, W).to(T) if c["gate"] else None
        st["grad_y"] = randn(R, W).to(T) if c["op"] == "norm_bwd" else None
        return st
    B, H, P, N, G = c["B"], c["H"], c["P"], c["N"], c["G"]
    step = c["op"] == "delta_step"
    rows = (B,) if step else (B, c["L"])
    # q, k, v come out of a conv with SiLU; dt and the beta logits out of a projection
    silu = lambda x: x * torch.sigmoid(x)  # noqa: E731
    if c["packed"]:
        vkq = silu(randn(*rows, H * P + 2 * G * N)).to(T)
        st["v"], st["k"], st["q"] = vkq[..., :H * P], vkq[..., H * P:H * P + G * N], vkq[..., H * P + G * N:]
    else:
        st["v"], st["k"], st["q"] = (silu(randn(*rows, n)).to(T) for n in (H * P, G * N, G * N))
    st["A"] = -torch.exp(rand(H) * math.log(16.0))
    st["dt_bias"] = -4.0 + 3.0 * rand(H)
    st["dt"], st["beta"] = randn(*rows, H), randn(*rows, H)
    if not c["raw"]:
        st["dt"], st["beta"] = torch.log1p(torch.exp(st["dt"] + st["dt_bias"])), torch.sigmoid(st["beta"])
        st["dt_bias"] = None
    if step:
        st["state"] = randn(B, H, P, N) * 0.3
        return st
    L = c["L"]
    st["init_state"] = randn(B, H, P, N) * 0.3 if c["state"] else None
    st["doc_ids"] = torch.cumsum((rand(B, L) < 1.0 / c["docs"]).int(), 1, dtype=torch.int32) if c["docs"] else None
    st["lengths"] = None
    if c["lengths"]:
        n = (rand(B) * (L + 1)).int()
        n[0] = L
        if B > 2:
            n[1] = 0
        st["lengths"] = n
    if c["op"] == "delta_bwd":
        st["grad_y"] = randn(B, L, H * P).to(T)
        st["grad_final_state"] = randn(B, H, P, N) * 0.3 if c["state"] else None
    return st


def run(st):
    return {"delta_fwd": _run_delta_fwd, "delta_step": _run_delta_step, "delta_bwd": _run_delta_bwd,
            "norm_fwd": _run_norm_fwd, "norm_bwd": _run_norm_bwd}[st["case"]["op"]](st)


# ------------------------------------------------------------------ the framework's calls
def _own_kw(st):
    c = st["case"]
    return dict(H=c["H"], P=c["P"], N=c["N"], G=c["G"], qk_norm=True, dt_softplus=c["raw"], dt_bias=st["dt_bias"],
                beta_sigmoid=c["raw"])


def _own_delta_fwd(st):
    import selective_state_space_14_amd as ssd
    c = st["case"]
    state = torch.empty(c["B"], c["H"], c["P"], c["N"], dtype=torch.float32, device=st["q"].device)
    y = ssd.ssd_delta_scan_fwd(st["q"], st["k"], st["v"], st["dt"], st["A"], st["beta"], doc_ids=st["doc_ids"],
                               lengths=st["lengths"], init_state=st["init_state"], final_state=state, **_own_kw(st))
    return {"y": y, "state": state}


def _own_delta_step(st):
    import selective_state_space_14_amd as ssd
    y = ssd.ssd_delta_step(st["q"], st["k"], st["v"], st["dt"], st["A"], st["beta"], st["state"], **_own_kw(st))
    return {"y": y, "state": st["state"]}


def _own_delta_bwd(st):
    import selective_state_space_14_amd as ssd
    g = ssd.ssd_delta_scan_bwd(st["q"], st["k"], st["v"], st["dt"], st["A"], st["beta"], st["grad_y"],
                               doc_ids=st["doc_ids"], lengths=st["lengths"], init_state=st["init_state"],
                               grad_final_state=st["grad_final_state"], **_own_kw(st))
    return {name: g[name] for name in ("q", "k", "v", "dt", "beta", "A", "dt_bias", "init_state") if name in g}


def _own_norm_fwd(st):
    import selective_state_space_14_amd as ssd
    return ssd.ssd_norm_fwd(st["x"], st["weight"], bias=st["bias"], z=st["z"], rms=st["case"]["rms"],
                            out_dtype=_dt(st["case"]["dtype"]))


def _own_norm_bwd(st):
    import selective_state_space_14_amd as ssd
    g = ssd.ssd_norm_bwd(st["x"], st["grad_y"], st["weight"], bias=st["bias"], z=st["z"], rms=st["case"]["rms"])
    return {name: g[name] for name in ("x", "weight", "bias", "z") if name in g}


# ------------------------------------------------------------------ the plain forms
def _gates(st):
    """dt after its softplus and beta after its sigmoid."""
    dt, beta = st["dt"], st["beta"]
    if st["case"]["raw"]:
        v = dt + st["dt_bias"]
        dt = torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-torch.abs(v)))
        beta = 1.0 / (1.0 + torch.exp(-beta))
    return dt, beta


def _chunks(st):
    """Everything that does not depend on the state, in blocks of CHUNK tokens: [B, H, blocks, CHUNK, ...]."""
    c = st["case"]
    B, L, H, P, N, G = (c[n] for n in ("B", "L", "H", "P", "N", "G"))
    n = -(-L // CHUNK)
    dev = st["q"].device
    live = torch.ones(B, L, dtype=torch.bool, device=dev)
    if st["lengths"] is not None:
        live = torch.arange(L, device=dev)[None] < st["lengths"][:, None]
    starts = torch.zeros(B, L, dtype=torch.int32, device=dev)
    if st["doc_ids"] is not None:
        starts[:, 1:] = (st["doc_ids"][:, 1:] != st["doc_ids"][:, :-1]).int()
    starts = starts * live

    def block(x):      # [B, L, H, ...] -> [B, H, n, CHUNK, ...]
        pad = torch.zeros((B, n * CHUNK) + x.shape[2:], dtype=x.dtype, device=dev)
        pad[:, :L] = x
        return pad.reshape((B, n, CHUNK) + x.shape[2:]).movedim(3, 1)

    def heads(x):      # a group's columns for each of its heads
        x = x.float().reshape(B, L, G, N) * live[..., None, None]
        return x.repeat_interleave(H // G, 2)

    dt, beta = _gates(st)
    d = {"n": n, "live": live}
    q, k = heads(st["q"]), heads(st["k"])
    rq, rk = (torch.rsqrt((x * x).sum(-1) + QK_EPS) for x in (q, k))
    d["rq"], d["rk"] = block(rq), block(rk)
    d["q"], d["k"] = block(q * rq[..., None]), block(k * rk[..., None])
    d["v"] = block(st["v"].float().reshape(B, L, H, P) * live[..., None, None])
    d["beta"] = block(beta * live[..., None])
    d["dt"] = block(dt * live[..., None])
    g = torch.cumsum(d["dt"].double() * st["A"].double()[None, :, None, None], -1)
    seg = torch.cumsum(block(starts[..., None].expand(B, L, H)), -1)
    same = (seg[..., :, None] == seg[..., None, :]).tril()
    d["M"] = torch.where(same, torch.exp(torch.clamp(g[..., :, None] - g[..., None, :], max=0.0)), 0.0).float()
    d["into"] = torch.where(seg == 0, torch.exp(g), 0.0).float()
    d["out"] = torch.where(seg == seg[..., -1:], torch.exp(g[..., -1:] - g), 0.0).float()
    d["across"] = torch.where(seg[..., -1] == 0, torch.exp(g[..., -1]), 0.0).float()
    d["KM"] = (d["k"] @ d["k"].transpose(-1, -2)) * d["M"].tril(-1)
    low = d["beta"][..., None] * d["KM"]
    inv = -low
    for i in range(1, CHUNK):
        inv[..., i, :i] += (inv[..., i, None, :i] @ inv[..., :i, :i])[..., 0, :]
    d["low"], d["inv"] = low, inv + torch.eye(CHUNK, device=dev)
    d["att"] = (d["q"] @ d["k"].transpose(-1, -2)) * d["M"] * N ** -0.5
    return d


def _first_state(st, d):
    c = st["case"]
    if st["init_state"] is None:
        return torch.zeros(c["B"], c["H"], c["N"], c["P"], device=st["q"].device)
    return st["init_state"].transpose(-1, -2)


def _through(st, d):
    """The blocks in turn: X = V - decay K S and U = (I + low)^-1 beta X of each, and the state before and after."""
    S, X, U, states = _first_state(st, d), [], [], []
    for i in range(d["n"]):
        states.append(S)
        X.append(d["v"][:, :, i] - d["into"][:, :, i, :, None] * (d["k"][:, :, i] @ S))
        U.append(d["inv"][:, :, i] @ (d["beta"][:, :, i, :, None] * X[i]))
        S = d["across"][:, :, i, None, None] * S + (d["k"][:, :, i] * d["out"][:, :, i, :, None]).transpose(-1, -2) @ U[i]
    stack = lambda v: torch.stack(v, 2)  # noqa: E731
    return stack(X), stack(U), stack(states), S


def _rows(st, x):
    """[B, H, blocks, CHUNK, ...] -> [B, L, H, ...]"""
    c = st["case"]
    return x.movedim(1, 3).flatten(1, 2)[:, :c["L"]]


def _run_delta_fwd(st):
    if own:
        return _own_delta_fwd(st)
    c, d = st["case"], _chunks(st)
    _, U, S, last = _through(st, d)
    y = c["N"] ** -0.5 * d["into"][..., None] * (d["q"] @ S) + d["att"] @ U
    y = _rows(st, y).reshape(c["B"], c["L"], c["H"] * c["P"])
    return {"y": y.to(st["v"].dtype), "state": last.transpose(-1, -2).contiguous()}


def _run_delta_step(st):
    if own:
        return _own_delta_step(st)
    c = st["case"]
    B, H, P, N, G = (c[n] for n in ("B", "H", "P", "N", "G"))
    dt, beta = _gates(st)
    q, k = (st[n].float().reshape(B, G, N).repeat_interleave(H // G, 1) for n in ("q", "k"))
    q, k = (x * torch.rsqrt((x * x).sum(-1, keepdim=True) + QK_EPS) for x in (q, k))
    S = st["state"] * torch.exp(dt * st["A"])[..., None, None]
    u = beta[..., None] * (st["v"].float().reshape(B, H, P) - (S * k[:, :, None]).sum(-1))
    S = S + u[..., None] * k[:, :, None]
    y = N ** -0.5 * (S * q[:, :, None]).sum(-1)
    st["state"].copy_(S)
    return {"y": y.reshape(B, H * P).to(st["v"].dtype), "state": st["state"]}


def _run_delta_bwd(st):
    if own:
        return _own_delta_bwd(st)
    c, d = st["case"], _chunks(st)
    B, L, H, P, N, G = (c[n] for n in ("B", "L", "H", "P", "N", "G"))
    n, T = d["n"], lambda x: x.transpose(-1, -2)  # noqa: E731
    X, U, S, last = _through(st, d)
    pad = torch.zeros(B, n * CHUNK, H, P, device=X.device)
    pad[:, :L] = st["grad_y"].float().reshape(B, L, H, P) * d["live"][..., None, None]
    dO = pad.reshape(B, n, CHUNK, H, P).movedim(3, 1)
    sO = N ** -0.5 * d["into"][..., None] * dO
    dS = torch.zeros_like(last) if st["grad_final_state"] is None else T(st["grad_final_state"])
    adj, Z = [None] * n, [None] * n
    for i in reversed(range(n)):
        adj[i] = dS
        dU = T(d["att"][:, :, i]) @ dO[:, :, i] + d["out"][:, :, i, :, None] * (d["k"][:, :, i] @ dS)
        Z[i] = T(d["inv"][:, :, i]) @ dU
        w = (d["beta"][:, :, i] * d["into"][:, :, i])[..., None]
        dS = d["across"][:, :, i, None, None] * dS + T(d["q"][:, :, i]) @ sO[:, :, i] - T(d["k"][:, :, i]) @ (w * Z[i])
    adj, Z = torch.stack(adj, 2), torch.stack(Z, 2)
    beta = d["beta"][..., None]
    dA_, dL = dO @ T(U), -(Z @ T(U))                        # of the attention and of the lower factor
    dbeta = (Z * X).sum(-1) + (dL * d["KM"]).sum(-1)
    pa, pl = dA_ * d["M"] * N ** -0.5, dL * d["M"].tril(-1) * beta
    q_in, k_in = sO @ T(S), -(beta * d["into"][..., None]) * (Z @ T(S))
    k_out = d["out"][..., None] * (U @ T(adj))
    dq = q_in + pa @ d["k"]
    dk = k_in + k_out + T(pa) @ d["q"] + pl @ d["k"] + T(pl) @ d["k"]
    ea, el = (dA_ * d["att"]).double(), (dL * d["low"]).double()
    out = (k_out * d["k"]).double().sum(-1)
    dG = ea.sum(-1) - ea.sum(-2) + el.sum(-1) - el.sum(-2) + ((q_in * d["q"]).double() + (k_in * d["k"]).double()).sum(-1) - out
    dG[..., -1] += out.sum(-1) + d["across"].double() * (S * adj).double().sum((-1, -2))
    dg = torch.flip(torch.cumsum(torch.flip(dG, [-1]), -1), [-1])
    res = {}
    for name, grad, unit, r in (("q", dq, d["q"], d["rq"]), ("k", dk, d["k"], d["rk"])):
        grad = (grad - unit * (unit * grad).sum(-1, keepdim=True)) * r[..., None]
        res[name] = _rows(st, grad).reshape(B, L, G, H // G, N).sum(3).reshape(B, L, G * N) * d["live"][..., None]
        res[name] = res[name].to(st[name].dtype)
    res["v"] = _rows(st, beta * Z).reshape(B, L, H * P).to(st["v"].dtype)
    res["A"] = (dg * d["dt"]).sum((0, 2, 3)).float()
    ddt = _rows(st, dg * st["A"].double()[None, :, None, None]) * d["live"][..., None]
    dbeta = _rows(st, dbeta) * d["live"][..., None]
    if c["raw"]:
        v = st["dt"] + st["dt_bias"]
        ddt = ddt / (1.0 + torch.exp(-v.double()))
        res["dt_bias"] = ddt.sum((0, 1)).float()
        s = 1.0 / (1.0 + torch.exp(-st["beta"]))
        dbeta = dbeta * s * (1.0 - s)
    res["dt"], res["beta"] = ddt.float(), dbeta
    if st["init_state"] is not None:
        res["init_state"] = T(dS).contiguous()
    return res


def _hat(st):
    x = st["x"].float()
    if not st["case"]["rms"]:
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5)
    return x * r, r


def _run_norm_fwd(st):
    if own:
        return _own_norm_fwd(st)
    y = _hat(st)[0] * st["weight"]
    if st["bias"] is not None:
        y = y + st["bias"]
    if st["z"] is not None:
        z = st["z"].float()
        y = y * (z / (1.0 + torch.exp(-z)))
    return y.to(_dt(st["case"]["dtype"]))


def _run_norm_bwd(st):
    if own:
        return _own_norm_bwd(st)
    hat, r = _hat(st)
    g, res = st["grad_y"].float(), {}
    if st["z"] is not None:
        z = st["z"].float()
        s = 1.0 / (1.0 + torch.exp(-z))
        n = hat * st["weight"]
        if st["bias"] is not None:
            n = n + st["bias"]
        res["z"] = (g * n * s * (1.0 + z * (1.0 - s))).to(st["z"].dtype)
        g = g * z * s
    res["weight"] = (g * hat).sum(0)
    if st["bias"] is not None:
        res["bias"] = g.sum(0)
    g = g * st["weight"]
    dx = g - hat * (g * hat).mean(-1, keepdim=True)
    if not st["case"]["rms"]:
        dx = dx - g.mean(-1, keepdim=True)
    res["x"] = (dx * r).to(st["x"].dtype)
    return res


# ------------------------------------------------------------------ the definition in 64 bits, token by token
def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"].startswith("norm"):
        return _exact_norm(c, st)
    B, H, P, N, G = (c[n] for n in ("B", "H", "P", "N", "G"))
    step, bwd = c["op"] == "delta_step", c["op"] == "delta_bwd"
    L = 1 if step else c["L"]
    if bwd and 8.0 * B * H * N * P * L > 60e9 or L > 60000:
        return None
    wide = lambda n, m: st[n].double().reshape(B, L, -1, m)  # noqa: E731
    own_head = torch.arange(H, device=st["q"].device) // (H // G)
    unit = lambda x: x / torch.sqrt((x ** 2).sum(-1, keepdim=True) + QK_EPS)  # noqa: E731
    q0, k0 = wide("q", N), wide("k", N)
    q, k, v = unit(q0)[:, :, own_head], unit(k0)[:, :, own_head], wide("v", P)
    raw_dt, raw_beta = st["dt"].double().reshape(B, L, H), st["beta"].double().reshape(B, L, H)
    dt, beta = raw_dt, raw_beta
    if c["raw"]:
        raw_dt = raw_dt + st["dt_bias"].double()
        dt, beta = torch.logaddexp(raw_dt, torch.zeros_like(raw_dt)), torch.sigmoid(raw_beta)
    A = st["A"].double()
    a = torch.exp(dt * A)
    fresh = torch.zeros(B, L, dtype=torch.bool, device=a.device)
    stop = torch.full((B,), L, device=a.device)
    if not step and st["doc_ids"] is not None:
        fresh[:, 1:] = st["doc_ids"][:, 1:] != st["doc_ids"][:, :-1]
    if not step and st["lengths"] is not None:
        stop = st["lengths"].long()
    live = torch.arange(L, device=a.device)[None] < stop[:, None]
    a = torch.where(live[..., None], torch.where(fresh[..., None], torch.zeros_like(a), a), torch.ones_like(a))
    beta = torch.where(live[..., None], beta, torch.zeros_like(beta))
    S = torch.zeros(B, H, P, N, dtype=torch.float64, device=a.device)
    first = st["state"] if step else st["init_state"]
    if first is not None:
        S = first.double()
    before, us = [], []
    ys = torch.zeros(B, L, H, P, dtype=torch.float64, device=a.device)
    for t in range(L):
        if bwd:
            before.append(S)
        S = S * a[:, t, :, None, None]
        kt = k[:, t, :, :, None]
        u = beta[:, t, :, None] * (v[:, t] - (S @ kt)[..., 0])
        S = S + u[..., None] * kt.transpose(-1, -2)
        if bwd:
            us.append(u)
        else:
            ys[:, t] = (S @ q[:, t, :, :, None])[..., 0] * N ** -0.5
    if not bwd:
        ys = torch.where(live[:, :, None, None], ys, torch.zeros_like(ys))
        return {"y": ys.reshape((B, H * P) if step else (B, L, H * P)), "state": S}
    gy = st["grad_y"].double().reshape(B, L, H, P) * live[..., None, None]
    gS = torch.zeros_like(S) if st["grad_final_state"] is None else st["grad_final_state"].double()
    gq, gk, gv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    ga, gb = torch.zeros_like(a), torch.zeros_like(beta)
    for t in reversed(range(L)):
        kt, u, old = k[:, t], us[t], before[t] * a[:, t, :, None, None]
        g = gy[:, t] * N ** -0.5
        gq[:, t] = (g[..., None, :] @ S)[..., 0, :]
        gS = gS + g[..., None] * q[:, t, :, None, :]
        gu = (gS @ kt[..., None])[..., 0]
        off = v[:, t] - (old @ kt[..., None])[..., 0]
        gb[:, t] = (gu * off).sum(-1)
        gv[:, t] = gu * beta[:, t, :, None]
        gk[:, t] = (u[..., None, :] @ gS)[..., 0, :] - (gv[:, t][..., None, :] @ old)[..., 0, :]
        gS = gS - gv[:, t][..., None] * kt[:, :, None, :]
        ga[:, t] = (gS * old).sum((-1, -2))            # times a: the gradient of dt A
        gS = gS * a[:, t, :, None, None]
        S = before[t]
    dead = ~live[..., None]
    ga, gb = ga.masked_fill(dead, 0.0), gb.masked_fill(dead, 0.0)
    res = {"v": gv.reshape(B, L, H * P), "A": (ga * dt).sum((0, 1)), "dt": ga * A, "beta": gb}
    for name, x, gr in (("q", q0, gq), ("k", k0, gk)):
        gr = gr.reshape(B, L, G, H // G, N).sum(3)
        size = torch.sqrt((x ** 2).sum(-1, keepdim=True) + QK_EPS)
        gr = gr / size - x * (x * gr).sum(-1, keepdim=True) / size ** 3
        res[name] = gr.reshape(B, L, G * N).masked_fill(dead, 0.0)
    if c["raw"]:
        res["dt"] = res["dt"] * torch.sigmoid(raw_dt)
        res["dt_bias"] = res["dt"].sum((0, 1))
        res["beta"] = gb * beta * (1.0 - beta)
    if st["init_state"] is not None:
        res["init_state"] = gS
    return res


def _exact_norm(c, st):
    bwd = c["op"] == "norm_bwd"
    leaf = lambda n: None if st[n] is None else st[n].double().requires_grad_(bwd)  # noqa: E731
    x, w, b, z = (leaf(n) for n in ("x", "weight", "bias", "z"))
    m = 0.0 if c["rms"] else x.sum(-1, keepdim=True) / c["W"]
    var = ((x - m) ** 2).sum(-1, keepdim=True) / c["W"]
    y = (x - m) / torch.sqrt(var + 1e-5) * w
    if b is not None:
        y = y + b
    if z is not None:
        y = y * z * torch.sigmoid(z)
    if not bwd:
        return y
    names = [n for n, t in (("x", x), ("weight", w), ("bias", b), ("z", z)) if t is not None]
    grads = torch.autograd.grad(y, [t for t in (x, w, b, z) if t is not None], st["grad_y"].double())
    return dict(zip(names, grads))


def work(case):
    c = case
    e = lambda name: 4 if name == "f32" else 2  # noqa: E731
    if c["op"].startswith("norm"):
        R, W, T, X = c["R"], c["W"], e(c["dtype"]), e(c["xdtype"])
        n = R * W
        par = 4 * W * (2 if c["bias"] else 1)
        if c["op"] == "norm_fwd":
            return {"bytes": n * (X + T + (T if c["gate"] else 0)) + par, "flops": 8 * n}
        return {"bytes": n * (2 * X + T + (2 * T if c["gate"] else 0)) + 2 * par, "flops": 16 * n}
    B, H, P, N, G, T = c["B"], c["H"], c["P"], c["N"], c["G"], e(c["dtype"])
    L = c.get("L", 1)
    tokens, S = B * L, 4 * B * H * P * N
    io = tokens * (T * (2 * G * N + H * P) + 8 * H) + (8 if c["raw"] else 4) * H
    if c["op"] == "delta_step":
        return {"bytes": io + T * tokens * H * P + 2 * S, "flops": 7 * tokens * H * P * N}
    if c["docs"]:
        io += 4 * tokens
    if c["op"] == "delta_fwd":
        return {"bytes": io + T * tokens * H * P + S * (2 if c["state"] else 1), "flops": 7 * tokens * H * P * N}
    return {"bytes": 2 * io + T * tokens * H * P + (3 * S if c["state"] else 0), "flops": 21 * tokens * H * P * N}
