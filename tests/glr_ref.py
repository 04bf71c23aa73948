"""64-bit reference of the gated linear recurrence, token by token on the CPU, with bounds of the kernels' errors.

Bounds, in units of U = 2^-24.  A sigmoid of v takes an exp2 of a rounded product, a sum and a reciprocal: (8 + 2|v|) U of
itself.  n = s|A| then is off by (10 + 2|v|) U, the decay a = e^-n by a n times that and two roundings, and
m = sqrt((1 - a)(1 + a)) by (16 + 2|v|) U of itself, since 1 - a is computed to a few U of itself.  The inputs m g x follow.
A state's error obeys the state's own recurrence: what each token adds is the error of its decay times the state before it,
the error of its input and the roundings of the steps and of the stretches' products, 4 U of the state's magnitude (the
recurrence of the inputs' magnitudes).  The adjoint's is the same in the other direction."""
from __future__ import annotations

import torch

F64, U = torch.float64, 2.0 ** -24


def masks(B, L, doc_ids=None, lengths=None):
    stop = torch.full((B,), L) if lengths is None else lengths.long().clamp(0, L)
    live = (torch.arange(L)[None] < stop[:, None])[..., None]
    fresh = torch.zeros(B, L, 1, dtype=torch.bool)
    if doc_ids is not None:
        fresh[:, 1:, 0] = doc_ids[:, 1:] != doc_ids[:, :-1]
    return live, fresh


def _through(a, b, first):
    """(states before, states after) every token of h <- a h + b."""
    h, before, after = first, [], []
    for t in range(a.shape[1]):
        before.append(h)
        h = a[:, t] * h + b[:, t]
        after.append(h)
    return torch.stack(before, 1), torch.stack(after, 1)


def glr(x, r, i, A, r_bias=None, i_bias=None, doc_ids=None, lengths=None, init_state=None, grad_y=None,
        grad_final_state=None):
    """({name: value}, {name: bound of its error before the last rounding}); the gradients where grad_y is given."""
    B, L, D = x.shape
    live, fresh = masks(B, L, doc_ids, lengths)
    # what stands behind a row's length is not used
    x, vr, vi = (torch.where(live, t.to(F64), torch.zeros((), dtype=F64)) for t in (x, r, i))
    vr = vr + (0 if r_bias is None else r_bias.to(F64))
    vi = vi + (0 if i_bias is None else i_bias.to(F64))
    A = A.to(F64)
    s, g = torch.sigmoid(vr), torch.sigmoid(vi)
    n = -s * A
    a, m = torch.exp(-n), torch.sqrt(-torch.expm1(-2 * n))
    one, zero = torch.ones((), dtype=F64), torch.zeros((), dtype=F64)
    keep = torch.where(live, torch.where(fresh, zero, a), one)
    b = torch.where(live, m * g * x, zero)
    wr, wi = vr.abs(), vi.abs()
    da = torch.where(live & ~fresh, a * (n * (12 + 2 * wr) + 2) * U, zero)
    # 1 - a^2 below the smallest normal number, 2^-126, may read as 0: its root is then off by up to 2^-63
    db = torch.where(live, b.abs() * (32 + 2 * wr + 2 * wi) * U + g * x.abs() * 2.0 ** -62, zero)
    first = torch.zeros(B, D, dtype=F64) if init_state is None else init_state.to(F64)
    before, after = _through(keep, b, first)
    mag0, mag = _through(keep, b.abs(), first.abs())
    err0, err = _through(keep, mag0 * da + db + 4 * U * mag, torch.zeros_like(first))
    val = {"y": torch.where(live, after, zero), "state": after[:, -1]}
    tol = {"y": torch.where(live, err, zero), "state": err[:, -1]}
    val["chunk_states"], tol["chunk_states"] = before[:, ::64], err0[:, ::64]
    if grad_y is None:
        return val, tol
    flip = lambda t: torch.flip(t, [1])  # noqa: E731
    gy = torch.where(live, grad_y.to(F64), zero)
    gf = torch.zeros_like(first) if grad_final_state is None else grad_final_state.to(F64)

    def back(own, last):
        """lam and what enters it from behind, keep_{t+1} lam_{t+1}; `last` enters the last token."""
        nu, lam, into = last, [], []
        for t in reversed(range(L)):
            into.append(nu)
            lam.append(own[:, t] + nu)
            nu = keep[:, t] * lam[-1]
        return flip(torch.stack(lam, 1)), flip(torch.stack(into, 1)), nu

    lam, _, out = back(gy, gf)
    lmag, _, omag = back(gy.abs(), gf.abs())
    after_da = torch.cat([da[:, 1:], torch.zeros_like(da[:, :1])], 1)
    after_lmag = torch.cat([lmag[:, 1:], torch.zeros_like(lmag[:, :1])], 1)
    lerr, _, oerr = back(after_lmag * after_da + 4 * U * lmag, torch.zeros_like(gf))
    val["init_state"], tol["init_state"] = out, oerr + lmag[:, 0] * da[:, 0] + 4 * U * omag
    cut = lambda t: torch.where(live, t, zero)  # noqa: E731
    safe = torch.where(m > 0, m, one)
    slope = torch.where(m > 0, a * a / safe, zero)
    dl = cut(lam * (keep * before - g * x * slope))
    ddl = cut(lerr * (keep * mag0 + g * x.abs() * slope)
              + lmag * (err0 * keep + mag0 * da + 2 * U * mag0 * keep + g * x.abs() * slope * (48 + 4 * wr + 2 * wi) * U))
    rel = (40 + 2 * wr + 2 * wi) * U
    val["x"], tol["x"] = cut(lam * m * g), cut(lerr * m * g + lmag * m * g * rel)
    val["i"] = cut(lam * m * x * g * (1 - g))
    tol["i"] = cut((lerr + lmag * rel) * m * x.abs() * g * (1 - g) + lmag * m * x.abs() * g * g * (8 + 2 * wi) * U)
    val["r"] = dl * A * s * (1 - s)
    tol["r"] = ddl * A.abs() * s * (1 - s) + dl.abs() * A.abs() * (s * (1 - s) * (16 + 4 * wr) + s * s * (8 + 2 * wr)) * U
    val["A"], tol["A"] = (dl * s).sum((0, 1)), (ddl * s + dl.abs() * s * (32 + 2 * wr) * U).sum((0, 1))
    for name, of in (("r_bias", "r"), ("i_bias", "i")):
        val[name], tol[name] = val[of].sum((0, 1)), (tol[of] + 20 * U * val[of].abs()).sum((0, 1))
    return val, tol
