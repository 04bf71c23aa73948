"""GPU: a row past 2^32 bytes of the delta scan.  As in test_gpu_delta_norm_large.py the last head is compared with a call of
its own: two bf16 calls, each within the scan tests' bounds of the exact result."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


def randn(*s, seed, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*s, generator=g, device=DEV, dtype=dtype)


def test_scan_and_its_backward(gpu_lib):
    """300,000 tokens of 128 heads: 4.9 GB of v and of y, 2.5 GB of q and of k."""
    B, L, H, P, N = 1, 300_000, 128, 64, 32
    q, k, v = (randn(B, L, n, seed=i, dtype=torch.bfloat16) for i, n in ((1, H * N), (2, H * N), (3, H * P)))
    dt, beta = randn(B, L, H, seed=5) - 2, randn(B, L, H, seed=6)
    A = -torch.exp(randn(H, seed=7))
    kw = dict(P=P, N=N, qk_norm=True, dt_softplus=True, beta_sigmoid=True)
    last = lambda t, n: t[-1:, :, -n:].contiguous()  # noqa: E731
    one = (last(q, N), last(k, N), last(v, P), last(dt, 1), A[-1:].clone(), last(beta, 1))
    fs, f1 = torch.empty(B, H, P, N, device=DEV), torch.empty(1, 1, P, N, device=DEV)

    def near(a, b, bound):
        a, b = a.double(), b.double()
        assert (a - b).norm() <= bound * b.norm(), float((a - b).norm() / b.norm())

    at = (slice(0, 64), slice(262_100, 262_200), slice(281_000, 282_000), slice(L - 100, L))
    y = gpu_lib.ssd_delta_scan_fwd(q, k, v, dt, A, beta, H=H, G=H, final_state=fs, **kw)
    y1 = gpu_lib.ssd_delta_scan_fwd(*one, H=1, G=1, final_state=f1, **kw)
    for s in at:
        near(y[-1, s, -P:], y1[0, s], 2.0 ** -5)
    near(fs[-1, -1], f1[0, 0], 2.0 ** -12)
    del y1
    gy = y                                           # as large, and no more memory
    g = gpu_lib.ssd_delta_scan_bwd(q, k, v, dt, A, beta, gy, H=H, G=H, **kw)
    g1 = gpu_lib.ssd_delta_scan_bwd(*one, last(gy, P), H=1, G=1, **kw)
    for name, n, bound in (("q", N, 2.0 ** -5), ("k", N, 2.0 ** -5), ("v", P, 2.0 ** -5), ("dt", 1, 2.0 ** -10), ("beta", 1, 2.0 ** -10)):
        for s in at:
            near(g[name][-1, s, -n:], g1[name][0, s], bound)
