"""GPU: ssd_add_norm_fwd and ssd_add_norm_bwd on rows off the 16-byte grid that a whole workgroup owns, more of them than workgroups, so
that each walks several: sums that meet in alternating places, rows fetched ahead, the weights' sums carried from row to row; and the
gradient in place of the stream's.  Bounds as in test_gpu_add_norm.py, whose checks these are."""
import pytest
import torch

from tests.test_gpu_add_norm import check_bwd, check_fwd, make, up

pytestmark = pytest.mark.gpu

# 256 threads a row (one and two vectors a thread) and 512; the forward's grid is 2048 workgroups, the backward's 1024
WIDTHS = [2079, 4095, 4097, 8191]


@pytest.mark.parametrize("t,rt,rms,gate", [("f32", "f32", False, True), ("bf16", "bf16", True, False), ("bf16", "f32", False, False)])
@pytest.mark.parametrize("W", WIDTHS)
def test_many_odd_rows(gpu_lib, W, t, rt, rms, gate):
    print(f"add_norm odd rows W={W} {t} {rt}", flush=True)
    d = make(2500, W, t, rt, t, gate=gate)
    check_fwd(gpu_lib, d, t, rms)
    a, g = check_bwd(gpu_lib, d, rt, t, rms), up(d)
    b = gpu_lib.ssd_add_norm_bwd(g["sum"], g["gy"], g["gs"], g["weight"], bias=g["bias"], z=g["z"], rms=rms)
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("W", [77, 1001, *WIDTHS])
def test_dsum_in_place_of_grad_sum(gpu_lib, W, t):
    """Through the C ABI's own arguments: a thread reads the vector that ends with the row, part of which its neighbours write."""
    lib, R, code = gpu_lib.load(), 2500, 0 if t == "f32" else 1
    d = make(R, W, t, t, t, bias=False)
    g = up(d)
    want = gpu_lib.ssd_add_norm_bwd(g["sum"], g["gy"], g["gs"], g["weight"], rms=True)
    dw = torch.empty(W, device=g["sum"].device)
    ws = torch.empty(gpu_lib.ssd_norm_bwd_workspace_size(R, 1, W), dtype=torch.uint8, device=g["sum"].device)
    st = lib.ssd_add_norm_bwd(R, W, code, code, 1, 1e-5, g["sum"].data_ptr(), W, g["weight"].data_ptr(), None, None, 0, g["gy"].data_ptr(), W,
                              g["gs"].data_ptr(), W, g["gs"].data_ptr(), W, dw.data_ptr(), None, None, 0, ws.data_ptr(), ws.numel(),
                              torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(g["gs"], want["sum"]) and torch.equal(dw, want["weight"])


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("W", WIDTHS)
def test_sum_in_place_of_the_residual(gpu_lib, W, t):
    d = make(2500, W, t, t, t)
    g = up(d)
    kw = dict(weight=g["weight"], bias=g["bias"], want_q=True)
    want = gpu_lib.ssd_add_norm_fwd(g["x"], g["residual"], **kw)
    for n in ("residual", "x"):
        h = {**g, n: g[n].clone()}
        got = gpu_lib.ssd_add_norm_fwd(h["x"], h["residual"], sum=h[n], **kw)
        assert torch.equal(h[n], want["sum"])
        assert all(torch.equal(got[k].view(torch.uint8), want[k].view(torch.uint8)) for k in want), n
