"""GPU: the backward of an empty batch: the gradients of the parameters, which have a size of their own, are zero."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV, H, P, N, G = "cuda", 8, 64, 64, 2


@pytest.fixture
def used_memory(gpu_lib):
    """The allocator's next small blocks held NaN before."""
    old = [torch.full((n,), float("nan"), device=DEV) for n in (H, 1024, 4096) for _ in range(16)]
    torch.cuda.synchronize()
    del old


def row(n, dtype=torch.float32):
    return torch.empty(0, 5, n, dtype=dtype, device=DEV)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_delta_scan_bwd(gpu_lib, used_memory, dtype):
    A, bias = -torch.ones(H, device=DEV), torch.zeros(H, device=DEV)
    g = gpu_lib.ssd_delta_scan_bwd(row(G * N, dtype), row(G * N, dtype), row(H * P, dtype), row(H), A, row(H),
                                   row(H * P, dtype), H=H, P=P, N=N, G=G, dt_softplus=True, dt_bias=bias,
                                   init_state=torch.empty(0, H, P, N, device=DEV))
    assert g["q"].shape == (0, 5, G * N) and g["init_state"].shape == (0, H, P, N)
    assert (g["A"] == 0).all() and (g["dt_bias"] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_scan_bwd(gpu_lib, used_memory, dtype):
    A, D, bias = (torch.ones(H, device=DEV) for _ in range(3))
    g = gpu_lib.ssd_chunk_scan_bwd(row(H * P, dtype), row(G * N, dtype), row(G * N, dtype), row(H), -A, row(H * P), H=H, P=P,
                                   N=N, G=G, D=D, dt_softplus=True, dt_bias=bias)
    assert g["x"].shape == (0, 5, H * P)
    assert all((g[n] == 0).all() for n in ("A", "D", "dt_bias"))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_mixer_bwd(gpu_lib, used_memory, dtype):
    C = H * P + 2 * G * N
    A, D, bias = (torch.ones(H, device=DEV) for _ in range(3))
    w, b = torch.ones(C, 4, device=DEV), torch.ones(C, device=DEV)
    g = gpu_lib.ssd_mixer_bwd(row(C, dtype), row(H, dtype), w, -A, row(H * P), H=H, P=P, N=N, G=G, conv_b=b, dt_bias=bias, D=D)
    assert g["raw"].shape == (0, 5, C)
    assert all((g[n] == 0).all() for n in ("A", "D", "dt_bias", "w", "bias"))
