"""GPU: the sums of ssd_delta_scan_bwd behind dt's, A's and dt_bias's gradients, fp32 inputs.

d(dt A) of a token sums the pairs (earlier token or entering state, later token or leaving gradient) across it; the kernel
takes it as row sums minus column sums, in which every pair on one side of the token cancels.  In 64 bits what is left of
those is 2^-53 for each addition a term passes, 34 at most (16 in a lane, 9 across lanes, 3 of a row's parts, 6 of the
running sum), of the sum of all terms' magnitudes M: below 2^-47 M."""
import pytest
import torch

from tests import delta_ref as ref
from tests.test_gpu_delta_bwd import cotangents, grads, wanted
from tests.test_gpu_delta_scan import make

pytestmark = pytest.mark.gpu

F64 = torch.float64


def magnitudes(d, opt, dims, gy, gS):
    """[B, H]: a bound of the sum of magnitudes of a chunk's terms, from the largest row of u and of its gradient, the
    largest state and the largest gradient of a state (q and k have length 1 at most, decays and beta are at most 1)."""
    H, P, N, G = dims
    B, L = d["q"].shape[:2]
    head = torch.arange(H) // (H // G)
    q, k = (ref.unit(d[n].to(F64).reshape(B, L, G, N), True)[:, :, head] for n in ("q", "k"))
    v, g = d["v"].to(F64).reshape(B, L, H, P), gy.to(F64).reshape(B, L, H, P) * N ** -0.5
    a, beta = torch.exp(d["dt"].to(F64) * d["A"].to(F64)), d["beta"].to(F64)
    S, D = opt["init_state"].to(F64), gS.to(F64)
    size = lambda x: x.flatten(2).norm(dim=-1)  # noqa: E731
    s = [size(S)]
    u, z, e = [], [], [size(D)]
    for t in range(L):
        S = S * a[:, t, :, None, None]
        r = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, None]).sum(-1))
        S = S + r[..., None] * k[:, t, :, None]
        u.append(size(r))
        s.append(size(S))
    for t in reversed(range(L)):
        D = D + g[:, t, ..., None] * q[:, t, :, None]
        r = (D * k[:, t, :, None]).sum(-1)
        D = (D - (beta[:, t, :, None] * r)[..., None] * k[:, t, :, None]) * a[:, t, :, None, None]
        z.append(size(r))
        e.append(size(D))
    u, z, s, e = (torch.stack(x).amax(0) for x in (u, z, s, e))
    rows = g.norm(dim=-1).amax(1)
    return 64 * 64 * (rows + z) * u + 64 * (rows + z) * s + 64 * u * e + s * e


@pytest.mark.parametrize("dims", [(2, 64, 32, 1), (2, 64, 64, 2), (1, 128, 128, 1)])
def test_a_strong_decay_leaves_no_residue(gpu_lib, dims):
    """Across a token of dt A = -25 every pair carries e^-25 (2^-36): the gradient there is that small, to the fp32 bound of
    the pairs themselves (2^-14), where sums in fp32 would leave 2^-24 of the terms on either side of the token."""
    d, opt = make(2, 140, *dims, torch.float32, state=True)
    H = dims[0]
    strong = [10, 40, 41, 63, 64, 100, 139]
    d["A"] = -torch.ones(H)
    d["dt"] = torch.full((2, 140, H), 0.02)
    d["dt"][:, strong] = 25.0
    d["beta"] = torch.sigmoid(d["beta"])
    gy, gS = cotangents(d, opt, dims)
    out = grads(gpu_lib, d, opt, dims, gy, gS, raw=False)
    want, _ = wanted(d, opt, dims, gy, gS, raw=False)
    M = magnitudes(d, opt, dims, gy, gS)[:, None]
    err = (out["dt"].double().cpu() - want["dt"]).abs()[:, strong]
    tol = (2.0 ** -46 + 2.0 ** -14 * 2.0 ** -36) * M
    assert (err <= tol).all(), float((err / tol).max())


def test_dt_bias_is_the_sum_of_dt(gpu_lib):
    """The tokens' gradients added in 64 bits and rounded once (2^-24)."""
    dims = (4, 64, 64, 2)
    d, opt = make(3, 500, *dims, torch.float32, state=True, lengths=[500, 333, 64])
    gy, gS = cotangents(d, opt, dims)
    out = grads(gpu_lib, d, opt, dims, gy, gS)
    dt = out["dt"].double().flatten(0, 1)
    err = (out["dt_bias"].double() - dt.sum(0)).abs()
    tol = 2.0 ** -24 * dt.sum(0).abs() + 2.0 ** -43 * dt.abs().sum(0)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("lengths", [None, [0, 1, 150]])
def test_nothing_passes_into_a_first_token(gpu_lib, dtype, state, lengths):
    """The gradient of dt at a document's first token, and at a row's where no state enters it, is exactly 0.  Of the
    other tokens it is not, a row's first with a state among them, where dt A > -5: the pairs across such a token carry 2^-8
    or more.  (Below dt A = -30 the kernel returns 0, and in between what pairs are left can round away.)"""
    dims = (2, 64, 64, 1)
    d, opt = make(3, 150, *dims, dtype, state=state, lengths=lengths, docs=0.05)
    opt["doc_ids"][:, 63:] += 1
    opt["doc_ids"][:, 64:] += 1                      # a document of one token at a chunk's end, one that starts a chunk
    gy, gS = cotangents(d, opt, dims)
    out = grads(gpu_lib, d, opt, dims, gy, gS)["dt"].cpu()
    first = torch.zeros(3, 150, dtype=torch.bool)
    first[:, 1:] = opt["doc_ids"][:, 1:] != opt["doc_ids"][:, :-1]
    first[:, 0] = not state
    assert (out[first] == 0).all(), out[first].abs().max()
    live = torch.arange(150)[None] < torch.tensor([150] * 3 if lengths is None else lengths)[:, None]
    dt, _ = ref.gates(d["dt"], d["beta"], True, d["dt_bias"], True)
    seen = (live & ~first)[..., None] & (dt * d["A"].double() > -5.0)
    assert seen[:, 0].any() == state and (out[seen] != 0).all()
