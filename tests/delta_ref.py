"""64-bit references of the gated delta rule and the row norm: the definitions, token by token, on the CPU.

`delta` also returns magnitudes (the same sums with absolute values) that the tests' error bounds are multiples of."""
from __future__ import annotations

import torch

F64 = torch.float64
QK_EPS = 1e-6


def unit(x, norm):
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + QK_EPS) if norm else x


def gates(dt, beta, softplus, dt_bias, sigmoid):
    dt, beta = dt.to(F64), beta.to(F64)
    if softplus:
        dt = dt + (0.0 if dt_bias is None else dt_bias.to(F64))
        dt = torch.logaddexp(dt, torch.zeros_like(dt))
    if sigmoid:
        beta = torch.sigmoid(beta)
    return dt, beta


def delta(q, k, v, dt, A, beta, *, H, P, N, G, scale=None, qk_norm=False, dt_softplus=False, dt_bias=None,
          beta_sigmoid=False, doc_ids=None, lengths=None, init_state=None):
    """(y [B, L, H*P], final state [B, H, P, N]) of [B, L, ...] inputs; differentiable in 64 bits."""
    B, L = q.shape[:2]
    scale = N ** -0.5 if scale is None else scale
    head = torch.arange(H) // (H // G)
    qh = unit(q.to(F64).reshape(B, L, G, N), qk_norm)[:, :, head]
    kh = unit(k.to(F64).reshape(B, L, G, N), qk_norm)[:, :, head]
    vh = v.to(F64).reshape(B, L, H, P)
    dt, beta = gates(dt, beta, dt_softplus, dt_bias, beta_sigmoid)
    A = A.to(F64)
    S = torch.zeros(B, H, P, N, dtype=F64) if init_state is None else init_state.to(F64)
    ys = []
    for t in range(L):
        on = torch.ones(B, dtype=torch.bool) if lengths is None else t < lengths
        a = torch.exp(dt[:, t] * A)
        if doc_ids is not None and t > 0:
            a = torch.where((doc_ids[:, t] != doc_ids[:, t - 1])[:, None], torch.zeros_like(a), a)
        M = S * a[..., None, None]
        u = beta[:, t, :, None] * (vh[:, t] - (M * kh[:, t, :, None]).sum(-1))
        M = M + u[..., None] * kh[:, t, :, None]
        y = scale * (M * qh[:, t, :, None]).sum(-1)
        m = on[:, None, None]
        ys.append(torch.where(m, y, torch.zeros_like(y)).reshape(B, H * P))
        S = torch.where(m[..., None], M, S)
    y = torch.stack(ys, 1) if ys else torch.zeros(B, 0, H * P, dtype=F64)
    return y, S


def norm(x, weight=None, bias=None, z=None, rms=False, eps=1e-5):
    x = x.to(F64)
    c = x if rms else x - x.mean(-1, keepdim=True)
    n = c / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    y = n if weight is None else n * weight.to(F64)
    if bias is not None:
        y = y + bias.to(F64)
    return y if z is None else y * torch.nn.functional.silu(z.to(F64))
