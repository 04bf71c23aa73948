"""GPU: the gated linear recurrence where numbers are not ordinary: NaN gates behind a document's start."""
import pytest
import torch

from tests.test_gpu_glr import DEV, bwd, fwd, make, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("L", [100, 2500])
def test_glr_nan_gates_behind_a_start(gpu_lib, t, L):
    """A NaN in r at a document's second token, or at any of its first ones, reaches no earlier document: neither their states
    and outputs nor, on the way back, their gradients and the initial state's.  Rows of two tiles and of many, starts at every
    place of a stretch of eight."""
    B, D = 2, 34
    d = make(B, L, D, t, state=True)
    g = to_dev(d)
    for start in [k for k in (1, 8, 17, 26, 35, 44, 53, 62, 71, 1503) if k < L]:
        ids = torch.zeros(B, L, dtype=torch.int32)
        ids[:, start:] = 1
        e = {**g, "doc_ids": ids.to(DEV)}
        clean, cleanb = fwd(gpu_lib, e), bwd(gpu_lib, e)
        for behind in (1, 2, 5, 7):
            e["r"] = g["r"].clone()
            e["r"][:, start + behind, ::3] = float("nan")
            out, back = fwd(gpu_lib, e), bwd(gpu_lib, e)
            assert torch.equal(out["y"][:, :start + behind], clean["y"][:, :start + behind]), (start, behind)
            assert torch.isnan(out["y"][:, start + behind:, ::3]).all(), (start, behind)
            for n in ("x", "r", "i"):
                assert torch.equal(back[n][:, :start], cleanb[n][:, :start]), (start, behind, n)
                other = [c for c in range(D) if c % 3]
                assert torch.equal(back[n][..., other], cleanb[n][..., other]), (start, behind, n)
                assert torch.isnan(back[n][:, start:start + behind + 1, ::3]).all(), (start, behind, n)
            assert torch.equal(back["init_state"], cleanb["init_state"]), (start, behind)
