"""GPU: operands past 2^31 bytes.  The far end of a large call is compared with a small call on copies of just that part:
bit for bit where the kernels choose the same order of sums, else within the two calls' bounds against 64 bits (the
delta scan's superchunks depend on the number of heads)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


def randn(*s, seed, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*s, generator=g, device=DEV, dtype=dtype)


def test_norm_rows(gpu_lib):
    R, W = 300_000, 4096                             # 2.46 GB of bf16
    x, z = randn(R, W, seed=1, dtype=torch.bfloat16), randn(R, W, seed=2, dtype=torch.bfloat16)
    w = randn(W, seed=3)
    y = gpu_lib.ssd_norm_fwd(x, w, z=z, rms=True)
    assert torch.equal(y[-50:], gpu_lib.ssd_norm_fwd(x[-50:].clone(), w, z=z[-50:].clone(), rms=True))
    g = gpu_lib.ssd_norm_bwd(x, y, w, z=z, rms=True)
    some = gpu_lib.ssd_norm_bwd(x[-50:].clone(), y[-50:].clone(), w, z=z[-50:].clone(), rms=True)
    assert torch.equal(g["x"][-50:], some["x"]) and torch.equal(g["z"][-50:], some["z"])


def test_step_state(gpu_lib):
    B, H, P, N, G = 1100, 64, 64, 128, 2             # 2.3 GB of state
    S = randn(B, H, P, N, seed=1)
    q, k, v = (randn(B, n, seed=i, dtype=torch.bfloat16) for i, n in ((2, G * N), (3, G * N), (4, H * P)))
    dt, beta = randn(B, H, seed=5), randn(B, H, seed=6)
    A = -torch.exp(randn(H, seed=7))
    kw = dict(H=H, P=P, N=N, G=G, qk_norm=True, dt_softplus=True, beta_sigmoid=True)
    few = S[-3:].clone()
    y = gpu_lib.ssd_delta_step(q, k, v, dt, A, beta, S, **kw)
    y3 = gpu_lib.ssd_delta_step(*(t[-3:].clone() for t in (q, k, v, dt)), A, beta[-3:].clone(), few, **kw)
    assert torch.equal(S[-3:], few) and torch.equal(y[-3:], y3)


def test_scan_and_its_backward(gpu_lib):
    """One row of 140,000 tokens and 128 heads, 2.3 GB of v; the last head against a call of its own.  Two bf16 calls, each
    within the scan tests' bounds of the exact result: their sum, 2^-5 for y and the gradients of q, k and v (2^-6 each),
    2^-10 for the fp32 outputs."""
    L, H, P, N = 140_000, 128, 64, 32
    q, k, v, gy = (randn(1, L, n, seed=i, dtype=torch.bfloat16) for i, n in ((1, H * N), (2, H * N), (3, H * P), (4, H * P)))
    dt, beta = randn(1, L, H, seed=5) - 2, randn(1, L, H, seed=6)
    A = -torch.exp(randn(H, seed=7))
    kw = dict(P=P, N=N, qk_norm=True, dt_softplus=True, beta_sigmoid=True)
    fs, f1 = torch.empty(1, H, P, N, device=DEV), torch.empty(1, 1, P, N, device=DEV)
    last = lambda t, n: t[..., -n:].contiguous()  # noqa: E731
    q1, k1, v1, dt1, b1, gy1 = last(q, N), last(k, N), last(v, P), last(dt, 1), last(beta, 1), last(gy, P)

    def near(a, b, bound):
        a, b = a.double(), b.double()
        assert (a - b).norm() <= bound * b.norm(), float((a - b).norm() / b.norm())

    y = gpu_lib.ssd_delta_scan_fwd(q, k, v, dt, A, beta, H=H, G=H, final_state=fs, **kw)
    y1 = gpu_lib.ssd_delta_scan_fwd(q1, k1, v1, dt1, A[-1:].clone(), b1, H=1, G=1, final_state=f1, **kw)
    for at in (slice(0, 64), slice(131_000, 136_000), slice(L - 100, L)):
        near(y[:, at, -P:], y1[:, at], 2.0 ** -5)
    near(fs[:, -1], f1[:, 0], 2.0 ** -12)
    del y, y1
    g = gpu_lib.ssd_delta_scan_bwd(q, k, v, dt, A, beta, gy, H=H, G=H, **kw)
    g1 = gpu_lib.ssd_delta_scan_bwd(q1, k1, v1, dt1, A[-1:].clone(), b1, gy1, H=1, G=1, **kw)
    for name, n, bound in (("q", N, 2.0 ** -5), ("k", N, 2.0 ** -5), ("v", P, 2.0 ** -5), ("dt", 1, 2.0 ** -10), ("beta", 1, 2.0 ** -10)):
        for at in (slice(0, 64), slice(131_000, 136_000), slice(L - 100, L)):
            near(g[name][:, at, -n:], g1[name][:, at], bound)
