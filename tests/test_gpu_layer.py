"""GPU: the operators of a recurrent layer in a row, as a model runs them: the norm with the residual's addition to 8 bits,
the projection to the recurrence's columns, the recurrence, its norm under a gate to 8 bits and the projection back, for a
ragged batch and then token by token; and the layer's gradients in training.

Every operator is held to its own bound at the values that it really got, and the whole to what no bound of a part shows:
that views fit together, that decoding goes on from the prefill's state, and that a captured run replays."""
import pytest
import torch

from tests import delta_ref, test_gpu_add_norm as add_norm, test_gpu_proj as proj
from tests.glr_ref import glr, masks

pytestmark = pytest.mark.gpu

DEV, E4M3 = "cuda", torch.float8_e4m3fn


def quantise(w):
    """[N, K] fp32 to e4m3 with a scale for every block of 128 by 128."""
    N, K = w.shape
    nb, kb = -(-N // 128), -(-K // 128)
    pad = torch.zeros(nb * 128, kb * 128)
    pad[:N, :K] = w
    scale = pad.view(nb, 128, kb, 128).abs().amax((1, 3)) / 448
    wide = scale.repeat_interleave(128, 0).repeat_interleave(128, 1)[:N, :K]
    return (w / wide).to(E4M3).to(DEV), scale.to(DEV)


def layer(W, D, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = dict(norm=1 + 0.2 * r(W), A=-torch.exp(torch.rand(D, generator=g) * 5 - 5), r_bias=0.5 * r(D), i_bias=0.5 * r(D), gated=1 + 0.2 * r(D))
    p = {n: v.to(DEV) for n, v in p.items()}
    p["up"], p["down"] = quantise(r(4 * D, W) / W ** 0.5), quantise(r(W, D) / D ** 0.5)
    return p


def mix(ssd, p, branch, stream, state, lengths=None, step=False, **out):
    """One layer over [B, L, W] (or one token, [B, W]): (its branch, the stream, what stood in between)."""
    D = p["A"].shape[0]
    n = ssd.ssd_add_norm_fwd(branch, stream, p["norm"], rms=True, out_dtype=torch.bfloat16, want_y=False, want_q=True, **out)
    u = ssd.ssd_proj_fp8_fwd(n["q"], n["scale"], *p["up"])
    x, r, i, z = (u[..., k * D:(k + 1) * D] for k in range(4))
    bias = dict(r_bias=p["r_bias"], i_bias=p["i_bias"])
    if step:
        y = ssd.ssd_glr_step(x, r, i, p["A"], state, **bias)
    else:
        y = ssd.ssd_glr_scan_fwd(x, r, i, p["A"], lengths=lengths, final_state=state, **bias)
    m = ssd.ssd_add_norm_fwd(y, weight=p["gated"], z=z, rms=True, want_y=False, want_q=True)
    return ssd.ssd_proj_fp8_fwd(m["q"], m["scale"], *p["down"]), n["sum"], dict(n=n, u=u, y=y, m=m)


def held(got, want, mag, name):
    """A value in its type against 64 bits: its own bound and half a step."""
    lim = mag + torch.finfo(got.dtype).eps / 2 * (want.abs() + mag) + 1e-30
    err = (got.double().cpu() - want).abs()
    assert (err <= lim).all(), (name, float((err / lim).max()))


def projected(got, q, scale, w, name):
    d = dict(a=q, a_scale=scale, w=w[0], w_scale=w[1])
    flat = {n: v.cpu().flatten(0, -2) for n, v in d.items()}
    want, mag = proj.reference(flat, "bf16")
    held(got.flatten(0, -2), want, mag, name)


def normed(n, s, weight, z, name):
    """q and its scale of the norm of s."""
    flat = lambda t: None if t is None else t.cpu().flatten(0, -2)  # noqa: E731
    s, z, w, W = flat(s), flat(z), weight.cpu(), s.shape[-1]
    want = delta_ref.norm(s, w, None, z, True)
    hat, _, off = add_norm.hat_parts(s, True)
    mag = (off + 4 * add_norm.U * hat.abs()) * w.double().abs()
    if z is not None:
        mag = mag * torch.nn.functional.silu(z.double()).abs() + (8 + 4 * z.double().abs()) * add_norm.U * want.abs()
    wide = flat(n["scale"]).double().repeat_interleave(128, 1)[:, :W]
    lim = mag * (1 + 2.0 ** -4) + (2.0 ** -4 + 8 * add_norm.U) * want.abs() + 2.0 ** -10 * wide
    assert ((flat(n["q"]).double() * wide - want).abs() <= lim).all(), name


def stages(p, branch, stream, out, mid, rows=None):
    """Every operator of a run but the recurrence; rows: the tokens that count, [B, L]."""
    of = (lambda t: t) if rows is None else (lambda t: t[rows])  # noqa: E731
    D = p["A"].shape[0]
    assert torch.equal(mid["n"]["sum"], (branch.float() + stream.float()).to(stream.dtype))
    normed({n: of(mid["n"][n]) for n in ("q", "scale")}, of(mid["n"]["sum"]), p["norm"], None, "the entry's norm")
    projected(of(mid["u"]), of(mid["n"]["q"]), of(mid["n"]["scale"]), p["up"], "the projection up")
    normed({n: of(mid["m"][n]) for n in ("q", "scale")}, of(mid["y"]), p["gated"], of(mid["u"][..., 3 * D:]), "the gated norm")
    projected(of(out), of(mid["m"]["q"]), of(mid["m"]["scale"]), p["down"], "the projection down")


@pytest.mark.parametrize("B,L,W,D", [(3, 150, 160, 144), (2, 600, 256, 400), (5, 9, 512, 80)])
def test_serving_a_ragged_batch(gpu_lib, B, L, W, D):
    print(f"layer B={B} L={L} W={W} D={D}", flush=True)
    ssd, p, more = gpu_lib, layer(W, D), 6
    g = torch.Generator().manual_seed(B * L)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    lengths = torch.randint(1, L + 1, (B,), generator=g, dtype=torch.int32)
    lengths[0] = L
    rows, _ = masks(B, L, None, lengths)
    rows = rows[..., 0].to(DEV)
    branch, stream = r(B, L, W), r(B, L, W)
    branch[~rows] = float("nan")                                    # what stands behind a sequence's end
    state = torch.empty(B, D, device=DEV)
    out, s, mid = mix(ssd, p, branch, stream, state, lengths.to(DEV))
    assert torch.isfinite(out[rows]).all() and torch.isfinite(state).all()
    keep = lambda t: torch.where(rows[..., None], t, 0)  # noqa: E731
    stages(p, keep(branch), stream, out, {**mid, "n": {**mid["n"], "sum": torch.where(rows[..., None], s, stream)}}, rows)
    columns = [mid["u"]]
    parts = [mid["y"]]
    for k in range(more):
        b1, s1 = r(B, W), r(B, W)
        o1, _, m1 = mix(ssd, p, b1, s1, state, step=True)
        stages(p, b1, s1, o1, m1)
        columns.append(m1["u"][:, None])
        parts.append(m1["y"][:, None])
    # every sequence as one: its prompt and the tokens after it, through the recurrence in 64 bits
    for b in range(B):
        n = int(lengths[b])
        u = torch.cat([columns[0][b, :n]] + [c[b] for c in columns[1:]])[None].cpu()
        val, tol = glr(u[..., :D], u[..., D:2 * D], u[..., 2 * D:3 * D], p["A"].cpu(), p["r_bias"].cpu(), p["i_bias"].cpu())
        y = torch.cat([parts[0][b, :n]] + [c[b] for c in parts[1:]])
        held(y, val["y"][0], tol["y"][0], "the recurrence")
        held(state[b], val["state"][0], tol["state"][0], "the state")


def test_decode_captured(gpu_lib):
    """Two layers' decode as a graph: a residual stream updated in place, states carried from replay to replay."""
    ssd, B, W, D = gpu_lib, 4, 256, 144
    ps = [layer(W, D, seed=s) for s in (1, 2)]
    g = torch.Generator().manual_seed(5)
    tokens = [torch.randn(2, B, W, generator=g).to(torch.bfloat16).to(DEV) for _ in range(4)]

    def token(branch, stream, states):
        for p, state in zip(ps, states):
            branch, stream, _ = mix(ssd, p, branch, stream, state, step=True, sum=stream)
        return branch

    states = [torch.randn(B, D, generator=g).to(DEV) for _ in ps]
    first = [s.clone() for s in states]
    want = []
    for t in tokens:
        s = t[1].clone()
        want.append((token(t[0], s, states), s, [v.clone() for v in states]))
    branch, stream, own = tokens[0][0].clone(), tokens[0][1].clone(), [s.clone() for s in first]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token(branch, stream, own)
    for again in range(2):
        for s, v in zip(own, first):
            s.copy_(v)
        for t, (o, s, v) in zip(tokens, want):
            branch.copy_(t[0])
            stream.copy_(t[1])
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, o) and torch.equal(stream, s) and all(torch.equal(a, b) for a, b in zip(own, v))


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ssd, x, residual, w):
        o = ssd.ssd_add_norm_fwd(x, residual, w, rms=True)
        ctx.ssd = ssd
        ctx.save_for_backward(o["sum"], w)
        return o["y"], o["sum"]

    @staticmethod
    def backward(ctx, gy, gs):
        s, w = ctx.saved_tensors
        g = ctx.ssd.ssd_add_norm_bwd(s, gy, gs, w, rms=True)
        return None, g["sum"], g["sum"], g["weight"]


class Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ssd, x, r, i, A, rb, ib, docs):
        B, L, D = x.shape
        cs = torch.empty(B, -(-L // 64), D, device=x.device)
        ctx.ssd = ssd
        ctx.save_for_backward(x, r, i, A, rb, ib, docs, cs)
        return ssd.ssd_glr_scan_fwd(x, r, i, A, r_bias=rb, i_bias=ib, doc_ids=docs, chunk_states=cs)

    @staticmethod
    def backward(ctx, gy):
        x, r, i, A, rb, ib, docs, cs = ctx.saved_tensors
        g = ctx.ssd.ssd_glr_scan_bwd(x, r, i, A, gy, r_bias=rb, i_bias=ib, doc_ids=docs, chunk_states=cs)
        return None, g["x"], g["r"], g["i"], g["A"], g["r_bias"], g["i_bias"], None


def plain(leaves, docs):
    """The training layer of test_training in 64 bits on the CPU, for autograd."""
    x, res, w, up, A, rb, ib, down = leaves
    s = x + res
    u = (s * torch.rsqrt((s * s).mean(-1, keepdim=True) + 1e-5) * w) @ up
    v, r, i = u.chunk(3, -1)
    a = torch.exp(torch.sigmoid(r + rb) * A)
    b = torch.sqrt(1 - a * a) * torch.sigmoid(i + ib) * v
    h, ys = torch.zeros_like(a[:, 0]), []
    for t in range(a.shape[1]):
        if t:
            h = torch.where((docs[:, t] != docs[:, t - 1])[:, None], torch.zeros_like(h), h)
        h = a[:, t] * h + b[:, t]
        ys.append(h)
    return torch.stack(ys, 1) @ down + s


def test_training(gpu_lib):
    """A layer's gradients in fp32 against autograd of the formula in 64 bits and against differences of it.

    Bound: every operator on the way (norm, product, recurrence and their backwards, six in all) is off by at most some 300
    units of 2^-24 of its terms' magnitudes (its own test), and no gain of this layer, whose maps are scaled to unit size
    and whose decays keep at most 1 / (1 - e^-0.02 / 2) < 100 tokens, but usually far fewer, lifts a norm by more than 32 on
    the way to a leaf: 6 * 300 * 32 * 2^-24 < 2^-8 of the gradient's norm."""
    ssd, B, L, W, D = gpu_lib, 2, 300, 96, 136
    g = torch.Generator().manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    leaves = [r(B, L, W), r(B, L, W), 1 + 0.2 * r(W), r(W, 3 * D) / W ** 0.5, -torch.exp(torch.rand(D, generator=g) * 4 - 3), 0.5 * r(D),
              0.5 * r(D), r(D, W) / D ** 0.5]
    docs = torch.cumsum((torch.rand(B, L, generator=g) < 0.02).int(), 1, dtype=torch.int32)
    gout = r(B, L, W)
    wide = [v.double().requires_grad_() for v in leaves]
    out = plain(wide, docs)
    want = torch.autograd.grad((out * gout.double()).sum(), wide)
    dev = [v.to(DEV).requires_grad_() for v in leaves]
    y, s = Norm.apply(ssd, dev[0], dev[1], dev[2])
    v, rr, i = (y @ dev[3]).chunk(3, -1)
    h = Recurrence.apply(ssd, v, rr, i, dev[4], dev[5], dev[6], docs.to(DEV))
    mine = h @ dev[7] + s
    got = torch.autograd.grad((mine * gout.to(DEV)).sum(), dev)
    close = lambda a, b: float((a.detach().double().cpu() - b).norm() / b.norm())  # noqa: E731
    assert close(mine, out.detach()) < 2.0 ** -8
    for k, (a, b) in enumerate(zip(got, want)):
        assert close(a, b) < 2.0 ** -8, (k, close(a, b))
    with torch.no_grad():
        loss = lambda moved: (plain(moved, docs) * gout.double()).sum()  # noqa: E731
        for k, v in enumerate(wide):
            d = r(*v.shape).double()
            d, e = d / d.norm(), 1e-5
            up, down = ([w + e * sign * d if j == k else w for j, w in enumerate(wide)] for sign in (1, -1))
            slope, own = float(loss(up) - loss(down)) / (2 * e), float((got[k].double().cpu() * d).sum())
            assert abs(slope - own) <= 2.0 ** -8 * float(want[k].norm()), (k, slope, own)
