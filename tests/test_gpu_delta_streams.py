"""GPU: the delta rule's and the norm's calls given a stream, and a sequence split captured into a graph."""
import pytest
import torch

from tests.test_gpu_delta_bwd import cotangents, grads
from tests.test_gpu_delta_scan import make, to_dev

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("handle", [False, True])
def test_given_a_stream(gpu_lib, handle):
    """What a call allocates belongs to the stream it is given: tensors that the current stream allocates and fills while
    the call still runs (as large as the workspace that is free again) change nothing."""
    ssd, (H, P, N, G) = gpu_lib, (8, 64, 64, 2)
    d, opt = make(2, 2000, H, P, N, G, torch.bfloat16, seed=1)
    gy, _ = cotangents(d, opt, (H, P, N, G), False)
    g, gy = to_dev(d), gy.to(DEV)
    kw = dict(H=H, P=P, N=N, G=G, qk_norm=True, dt_softplus=True, dt_bias=g["dt_bias"], beta_sigmoid=True)
    args = [g[n] for n in ("q", "k", "v", "dt", "A", "beta")]
    tok = [t[:, 0].contiguous() for t in args[:4]] + [g["A"], g["beta"][:, 0].contiguous()]
    x, w = torch.randn(3000, 2048, device=DEV), torch.randn(2048, device=DEV)
    state = torch.zeros(2, H, P, N, device=DEV)
    calls = [lambda **s: {"y": ssd.ssd_delta_scan_fwd(*args, **kw, **s)}, lambda **s: ssd.ssd_delta_scan_bwd(*args, gy, **kw, **s),
             lambda **s: {"y": ssd.ssd_delta_step(*tok, state.zero_() if not s else state, **kw, **s)},
             lambda **s: {"y": ssd.ssd_norm_fwd(x, w, **s)}, lambda **s: ssd.ssd_norm_bwd(x, x, w, **s)]
    sizes = [ssd.ssd_delta_scan_workspace_size(2, 2000, H, P, N, G), ssd.ssd_delta_scan_bwd_workspace_size(2, 2000, H, P, N, G),
             1024, 1024, ssd.ssd_norm_bwd_workspace_size(3000, 1, 2048)]
    for call, size in zip(calls, sizes):
        want = call()
        state.zero_()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        got = call(stream=side.cuda_stream if handle else side)
        over = [torch.full((max(n, 16) // 4,), float("nan"), device=DEV) for n in (size, *(t.nbytes for t in got.values()))]
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], want[n]) for n in want), call
        del over


def test_split_in_a_graph(gpu_lib):
    """Forward and backward of a sequence in superchunks, captured and replayed with new inputs between eager calls."""
    ssd, dims = gpu_lib, (1, 64, 64, 1)
    H, P, N, G = dims
    sets = [make(1, 1500, *dims, torch.bfloat16, seed=s) for s in range(3)]
    cots = [cotangents(d, o, dims, False, seed=i)[0] for i, (d, o) in enumerate(sets)]
    kw = lambda g: dict(H=H, P=P, N=N, G=G, qk_norm=True, dt_softplus=True, dt_bias=g["dt_bias"], beta_sigmoid=True)  # noqa: E731
    six = lambda g: [g[n] for n in ("q", "k", "v", "dt", "A", "beta")]  # noqa: E731
    want = []
    for (d, o), gy in zip(sets, cots):
        g = to_dev(d)
        want.append((ssd.ssd_delta_scan_fwd(*six(g), **kw(g)), grads(ssd, d, o, dims, gy, None)))
    g, gy = to_dev(sets[0][0]), cots[0].to(DEV)
    ws = torch.empty(max(ssd.ssd_delta_scan_workspace_size(1, 1500, H, P, N, G),
                         ssd.ssd_delta_scan_bwd_workspace_size(1, 1500, H, P, N, G)), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ssd.ssd_delta_scan_fwd(*six(g), workspace=ws, **kw(g))
        back = ssd.ssd_delta_scan_bwd(*six(g), gy, workspace=ws, **kw(g))
    for i in (1, 2, 0):
        for n, v in sets[i][0].items():
            g[n].copy_(v)
        gy.copy_(cots[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i][0]) and all(torch.equal(back[n], want[i][1][n]) for n in back)
        assert torch.equal(ssd.ssd_delta_scan_fwd(*six(g), workspace=ws, **kw(g)), want[i][0])
