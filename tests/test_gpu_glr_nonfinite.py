"""GPU: the gated linear recurrence where numbers are not ordinary: NaN gates behind a document's start, decays so near 1 that
1 - a^2 is subnormal, and infinite parameters."""
import pytest
import torch

from tests.test_gpu_glr import DEV, bwd, fwd, make, to_dev

pytestmark = pytest.mark.gpu

PARAMS = ("A", "r_bias", "i_bias")


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


def test_glr_subnormal_one_minus_square(gpu_lib):
    """0 < 1 - a^2 < 2^-126: its square root and the derivative of that are taken as 0, so dx and di are 0 there, all gradients
    finite, and what the token adds to dA is only what its decay of the held state gives.

    Tokens within a factor 2 of the border, or whose gate is itself below the smallest normal number, may go either way and are
    held to being finite (the sums are compared in channels without such tokens).  Bound of the others: glr_ref's terms at
    |v| <= 90, at most (48 + 4 * 90 + 32) * 2^-24 of the terms' magnitudes, and 2^-23 once more of decays that are subnormal
    themselves: below 2^-14."""
    B, L, D = 2, 100, 9
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    d = dict(x=r(B, L, D), i=r(B, L, D), r=r(B, L, D), grad_y=r(B, L, D), init_state=r(B, D), grad_final_state=r(B, D), r_bias=None,
             i_bias=None, doc_ids=None, lengths=None)
    d["A"] = torch.tensor([-0.002, -0.002, -0.5, -1.0, -1e-3, -1e-38, -2e-39, -4e-39, -1.5e-38])
    d["r"][..., 0] = -torch.arange(L) * 0.12 - 78.0                   # -78 .. -90
    d["r"][..., 1] = torch.where(torch.arange(L) % 9 == 4, -84.0, d["r"][..., 1])
    d["r"][..., 2:5] = -80.0 - 4.0 * torch.rand(B, L, 3, generator=gen)
    d["r"][..., 5:] *= 0.1                                          # gates near a half
    wide = {n: v.double() for n, v in d.items() if v is not None}
    s, g = torch.sigmoid(wide["r"]), torch.sigmoid(wide["i"])
    n = -s * wide["A"]
    a, m = torch.exp(-n), torch.sqrt(-torch.expm1(-2 * n))
    tiny = 2.0 ** -126
    zero, fine = (s >= 2 * tiny) & (2 * n < tiny / 2), (s >= 2 * tiny) & (2 * n > 2 * tiny)
    assert zero.sum() > 300 and (fine & (2 * n < 2.0 ** -100)).sum() > 300
    m = torch.where(zero, 0.0, m)
    slope = torch.where(m > 0, a * a / m.clamp_min(1e-300), 0.0)
    before, lam, h, nu = torch.empty_like(a), torch.empty_like(a), wide["init_state"], wide["grad_final_state"]
    for k in range(L):
        before[:, k] = h
        h = a[:, k] * h + m[:, k] * g[:, k] * wide["x"][:, k]
    for k in reversed(range(L)):
        lam[:, k] = wide["grad_y"][:, k] + nu
        nu = a[:, k] * lam[:, k]
    gx = g * wide["x"]
    dl = lam * (a * before - gx * slope)
    # magnitudes: of the adjoint and of the state, each a sum of at most L + 1 terms
    lmag = torch.flip(torch.cumsum(torch.flip(wide["grad_y"].abs(), [1]), 1), [1]) + wide["grad_final_state"].abs()[:, None]
    hmag = torch.cumsum((m * gx).abs(), 1) + wide["init_state"].abs()[:, None]
    rel = 2.0 ** -14
    want = dict(x=lam * m * g, i=lam * m * gx * (1 - g), r=dl * wide["A"] * s * (1 - s))
    dmag = lmag * (hmag + gx.abs() * slope)
    tol = dict(x=rel * lmag * m * g, i=rel * lmag * m * gx.abs(), r=rel * dmag * wide["A"].abs() * s)
    e = to_dev(d)
    none = zero.all(1).all(0).to(DEV)                                 # nothing is taken in: from a zero state nothing comes out
    assert none.sum() >= 2 and (fwd(gpu_lib, {**e, "init_state": None})["y"][..., none] == 0).all()
    y = fwd(gpu_lib, e)
    back = {n: v.double().cpu() for n, v in bwd(gpu_lib, e, chunk_states=y["chunk_states"]).items()}
    assert all(torch.isfinite(v).all() for v in back.values())
    assert (back["x"][zero] == 0).all() and (back["i"][zero] == 0).all()
    either = zero | fine
    for k in ("x", "i", "r"):
        off = (back[k] - want[k]).abs() <= tol[k] + 2.0 ** -120
        assert off[either].all(), (k, int((~off & either).sum()))
    whole = either.all(1).all(0)
    assert whole.sum() >= 2
    lim = (rel * dmag * s).sum((0, 1)) + 2.0 ** -120
    assert ((back["A"] - (dl * s).sum((0, 1))).abs() <= lim)[whole].all()


def test_glr_infinite_parameters(gpu_lib):
    """A of -inf (or so large that A log2 e is) forgets everything at each token, and biases of +-inf hold a gate open or shut:
    the same as large finite values give, behind a row's length too, where the state stops and gradients are 0."""
    inf = float("inf")
    for t, L in (("f32", 150), ("bf16", 150), ("bf16", 1500), ("f32", 900)):
        d = make(4, L, 14, t, state=True)
        d["lengths"] = torch.tensor([L, 0, L // 2, 3], dtype=torch.int32)
        live = torch.arange(L)[None] < d["lengths"][:, None]
        large = {n: d[n].clone() for n in PARAMS}
        for c, (n, v, w) in enumerate((("A", -inf, -1e30), ("A", -3e38, -1e30), ("r_bias", inf, 1e4), ("r_bias", -inf, -1e4), ("i_bias", inf, 1e4),
                                       ("i_bias", -inf, -1e4), ("r_bias", inf, 1e4))):
            d[n][2 * c], large[n][2 * c] = v, w
        d["A"][12] = large["A"][12] = -0.5
        e, f = to_dev(d), to_dev({**d, **large})
        for got, want in ((fwd(gpu_lib, e), fwd(gpu_lib, f)), (bwd(gpu_lib, e), bwd(gpu_lib, f))):
            for n in want:
                assert torch.isfinite(want[n]).all() and (got[n] == want[n]).all(), (t, L, n)
        back = bwd(gpu_lib, e)
        assert all((back[n].cpu()[~live] == 0).all() for n in ("x", "r", "i"))
        assert torch.equal(fwd(gpu_lib, e)["state"][1], e["init_state"][1])
        rows = [e[n][:, 0].contiguous() for n in ("x", "r", "i")]
        one, two = e["init_state"].clone(), e["init_state"].clone()
        kw = lambda p: dict(r_bias=p["r_bias"], i_bias=p["i_bias"])  # noqa: E731
        assert (gpu_lib.ssd_glr_step(*rows, e["A"], one, **kw(e)) == gpu_lib.ssd_glr_step(*rows, f["A"], two, **kw(f))).all()
        assert torch.isfinite(one).all() and (one == two).all()
