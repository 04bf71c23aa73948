"""GPU: ssd_delta_step against the definition in 64 bits.

Bounds.  A row's dot products are trees of N <= 128 terms (4 in a lane, up to 5 levels): 16 roundings of 2^-24 of the
sum of magnitudes cover them with the products before and after; the decay exp(dt A) is off by 2^-24 (4 + |dt A|) and
the softplus and sigmoid by a few 2^-24 more.  With m = |v| + a sum|S k| the new state is off by at most
c (a |S| + beta m |k|), and y by c scale sum |q| (a |S| + beta m |k|), c = 2^-24 (48 + 4 |dt A|), and then rounded."""
import pytest
import torch

from tests import delta_ref as ref

pytestmark = pytest.mark.gpu

DEV, U = "cuda", 2.0 ** -24


def make(B, H, P, N, G, dtype, packed=True, seed=0):
    g = torch.Generator().manual_seed(seed + B + 7 * H + N)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    HP, GN = H * P, G * N
    if packed:
        row = r(B, HP + 2 * GN).to(dtype)
        v, k, q = row[:, :HP], row[:, HP:HP + GN], row[:, HP + GN:]
    else:
        v, k, q = r(B, HP).to(dtype), r(B, GN).to(dtype), r(B, GN).to(dtype)
    return dict(q=q, k=k, v=v, dt=r(B, H), A=-torch.exp(2.7 * torch.rand(H, generator=g)), beta=r(B, H),
                dt_bias=r(H) - 2, state=r(B, H, P, N))


def check(ssd, d, H, P, N, G, raw=True, qk_norm=True, scale=None):
    B, T = d["q"].shape[0], d["q"].dtype
    g = {n: v.to(DEV) for n, v in d.items()}
    kw = dict(H=H, P=P, N=N, G=G, scale=scale, qk_norm=qk_norm, dt_softplus=raw, beta_sigmoid=raw)
    if not raw:
        g["dt"], g["beta"] = g["dt"].abs(), torch.sigmoid(g["beta"])
        d = {**d, "dt": g["dt"].cpu(), "beta": g["beta"].cpu()}
    bias = d["dt_bias"] if raw else None
    y = ssd.ssd_delta_step(g["q"], g["k"], g["v"], g["dt"], g["A"], g["beta"], g["state"],
                           dt_bias=g["dt_bias"] if raw else None, **kw)
    one = lambda n: d[n][:, None]  # noqa: E731
    wy, ws = ref.delta(one("q"), one("k"), one("v"), one("dt"), d["A"], one("beta"), dt_bias=bias,
                       init_state=d["state"], **kw)
    dt, beta = ref.gates(d["dt"], d["beta"], raw, bias, raw)
    e = dt * d["A"].double()
    head = torch.arange(H) // (H // G)
    q, k = (ref.unit(d[n].double().reshape(B, G, N), qk_norm)[:, head].abs() for n in ("q", "k"))
    aS = torch.exp(e)[..., None, None] * d["state"].double().abs()
    m = beta[..., None] * (d["v"].double().reshape(B, H, P).abs() + (aS * k[:, :, None]).sum(-1))
    c = U * (48 + 4 * e.abs())
    mag = aS + m[..., None] * k[:, :, None]
    tol = c[..., None, None] * mag
    err = (g["state"].double().cpu() - ws).abs()
    assert (err <= tol).all(), ("state", err.max(), (err / tol).max())
    s = abs(N ** -0.5 if scale is None else scale)
    tol = (c[..., None] * s * (mag * q[:, :, None]).sum(-1)).reshape(B, H * P)
    wy = wy[:, 0]
    tol = tol + torch.finfo(T).eps / 2 * (wy.abs() + tol)
    err = (y.double().cpu() - wy).abs()
    assert y.dtype == T and (err <= tol).all(), ("y", err.max(), (err / tol).max())
    return y, g["state"]


@pytest.mark.parametrize("B,H,P,N,G", [(1, 1, 64, 32, 1), (1, 32, 64, 64, 8), (3, 6, 128, 128, 2), (5, 4, 128, 32, 4),
                                       (130, 16, 64, 128, 1), (70, 12, 64, 64, 3), (260, 8, 128, 64, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_step(gpu_lib, B, H, P, N, G, dtype):
    print(f"delta_step B={B} H={H} P={P} N={N} G={G} {dtype}", flush=True)
    check(gpu_lib, make(B, H, P, N, G, dtype), H, P, N, G)
    check(gpu_lib, make(B, H, P, N, G, dtype, packed=False, seed=9), H, P, N, G, raw=False, qk_norm=False, scale=0.37)


def test_step_extreme_gates(gpu_lib):
    """Decays of 0 and 1, beta of 0 and 1, zero k and q rows (the norm's epsilon keeps them finite)."""
    d = make(4, 4, 64, 64, 2, torch.float32)
    d["dt"][0], d["dt"][1] = 200.0, -200.0
    d["beta"][2], d["beta"][3] = -200.0, 200.0
    d["k"][1], d["q"][2] = 0.0, 0.0
    check(gpu_lib, d, 4, 64, 64, 2)


def test_step_rows_do_not_depend_on_the_batch(gpu_lib):
    """One row alone and in a large batch (another number of rows a thread): the same bits."""
    H, P, N, G = 8, 64, 128, 2
    d = make(300, H, P, N, G, torch.bfloat16)
    y, s = check(gpu_lib, d, H, P, N, G)
    d1 = {n: v if n in ("A", "dt_bias") else v[17:18] for n, v in d.items()}
    y1, s1 = check(gpu_lib, d1, H, P, N, G)
    assert torch.equal(y1[0], y[17]) and torch.equal(s1[0], s[17])


def test_step_captured_and_replayed(gpu_lib):
    ssd, (H, P, N, G) = gpu_lib, (4, 64, 64, 2)
    d = {n: v.to(DEV) for n, v in make(6, H, P, N, G, torch.bfloat16).items()}
    first = d["state"].clone()
    call = lambda st: ssd.ssd_delta_step(d["q"], d["k"], d["v"], d["dt"], d["A"], d["beta"], st, H=H, P=P, N=N, G=G,  # noqa: E731
                                         qk_norm=True, dt_softplus=True, dt_bias=d["dt_bias"], beta_sigmoid=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(d["state"])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call(d["state"])
    d["state"].copy_(first)
    eager = first.clone()
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        want = call(eager)
        assert torch.equal(y, want) and torch.equal(d["state"], eager)
