"""GPU: ssd_norm_fwd and ssd_norm_bwd without an epsilon, where rows do not fill a workgroup.

Bounds as in test_gpu_norm.py: 64 roundings of 2^-24 for a pass of sums over a row, and 64 + R of them for a column's sum
over R rows; x has a mean of 0.5 and a deviation of 2, and at W = 1 only the rms norm divides by anything."""
import pytest
import torch

from tests import delta_ref as ref

pytestmark = pytest.mark.gpu

DEV, U = "cuda", 2.0 ** -24
# rows of a workgroup and a row width for each number of threads a row up to a wave's, read in vectors and one by one
ROWS = [(32, 64), (16, 128), (8, 256), (4, 512), (4, 1024), (4, 2048), (16, 1), (16, 15), (4, 63), (4, 201), (4, 777), (1, 3000)]


@pytest.mark.parametrize("rows,W", ROWS)
@pytest.mark.parametrize("gate", [False, True])
def test_no_epsilon(gpu_lib, rows, W, gate):
    for R in sorted({1, max(1, rows - 1), rows, rows + 1, 3 * rows + 1}):
        for rms in (True,) if W == 1 else (False, True):
            print(f"norm eps=0 R={R} W={W} rms={rms} gate={gate}", flush=True)
            gen = torch.Generator().manual_seed(R + 7 * W)
            r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
            d = dict(x=2 * r(R, W) + 0.5, weight=1 + 0.3 * r(W), bias=0.3 * r(W), z=r(R, W) if gate else None)
            gy = r(R, W)
            dev = {n: None if v is None else v.to(DEV) for n, v in d.items()}
            y = gpu_lib.ssd_norm_fwd(dev["x"], dev["weight"], bias=dev["bias"], z=dev["z"], rms=rms, eps=0.0)
            out = gpu_lib.ssd_norm_bwd(dev["x"], gy.to(DEV), dev["weight"], bias=dev["bias"], z=dev["z"], rms=rms, eps=0.0)
            leaf = {n: v.double().requires_grad_() for n, v in d.items() if v is not None}
            wy = ref.norm(leaf["x"], leaf["weight"], leaf["bias"], leaf.get("z"), rms, 0.0)
            want = dict(zip(leaf, torch.autograd.grad(wy, list(leaf.values()), gy.double())))
            assert set(out) == set(want) and torch.isfinite(y).all() and all(torch.isfinite(v).all() for v in out.values())
            x = d["x"].double()
            c = x if rms else x - x.mean(-1, keepdim=True)
            rstd = 1 / torch.sqrt((c * c).mean(-1, keepdim=True))
            n = c * rstd
            off = 64 * U * (2 * n.abs() + (0 if rms else x.abs().mean(-1, keepdim=True) * rstd))
            s = torch.nn.functional.silu(d["z"].double()) if gate else torch.ones(())
            rel = (16 + 4 * d["z"].double().abs()) * U if gate else 4 * U
            tol = (off * d["weight"].double().abs() + (8 * U + rel) * (n.abs() * d["weight"].double().abs() + d["bias"].double().abs())) * s.abs()
            assert ((y.double().cpu() - wy).abs() <= tol + 1e-30).all()
            g = (gy.double() * s).abs()
            for name, t in (("weight", (g * (n.abs() * ((64 + R) * U + rel) + off)).sum(0)),
                            ("bias", (g * ((64 + R) * U + rel)).sum(0))):
                err = (out[name].double().cpu() - want[name]).abs()
                assert (err <= t + 1e-30).all(), (name, float((err - t).max()))
            gw = g * d["weight"].double().abs()
            m1, m2 = gw.mean(-1, keepdim=True), (gw * n.abs()).mean(-1, keepdim=True)
            tol = rstd * (gw * (rel + 8 * U) + (64 * U + (rel * gw).mean(-1, keepdim=True) / (m1 + 1e-300)) * (m1 + n.abs() * m2)
                          + off * m2 + n.abs() * (gw * off).mean(-1, keepdim=True)) + 128 * U * want["x"].abs() + U * want["x"].abs()
            err = (out["x"].double().cpu() - want["x"]).abs()
            assert (err <= tol).all(), ("x", float((err - tol).max()))
