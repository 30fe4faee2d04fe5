"""Plain 64-bit forms of the decoder operators around the Gated Residual, from their definitions (CPU)."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24    # unit roundoff of fp32
UBF = 2.0 ** -8     # of bf16


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64)


def embed_grad(dR, ids, V, scale):
    """(gradient, sum of magnitudes, rows added) per table row."""
    rows = f64(dR)
    rows = rows if rows.dim() == 2 else rows.sum(1)
    mags = f64(dR).abs()
    mags = mags if mags.dim() == 2 else mags.sum(1)
    ids = ids.cpu().long()
    ok = (ids >= 0) & (ids < V)
    D = rows.shape[1]
    g = torch.zeros(V, D, dtype=torch.float64).index_add_(0, ids[ok], rows[ok]) * scale
    m = torch.zeros(V, D, dtype=torch.float64).index_add_(0, ids[ok], mags[ok]) * abs(scale)
    return g, m, torch.bincount(ids[ok], minlength=V).double()[:, None]


def layer_norm(x, w, b, eps):
    x = f64(x)
    mean = x.mean(-1)
    c = x - mean[..., None]
    rstd = 1 / (c.square().mean(-1) + eps).sqrt()
    xh = c * rstd[..., None]
    y = xh * f64(w)
    return y if b is None else y + f64(b), mean, rstd, xh


def layer_norm_grad(dy, x, w, mean, rstd):
    dy, r = f64(dy), f64(rstd)[..., None]
    xh = (f64(x) - f64(mean)[..., None]) * r
    u = dy * f64(w)
    m2 = (u * xh).mean(-1, keepdim=True)
    dx = r * (u - u.mean(-1, keepdim=True) - xh * m2)
    size = r * (u.abs() + u.abs().mean(-1, keepdim=True) + xh.abs() * (u * xh).abs().mean(-1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0), size, (dy * xh).abs().sum(0), dy.abs().sum(0)


def recurrence(q, k, v, log_decay, scale, starts, state=None, magnitudes=False):
    """o and the last states, token by token; with magnitudes the same sums of absolute values."""
    q, k, v, lam = f64(q), f64(k), f64(v), torch.exp(f64(log_decay))
    if magnitudes:
        q, k, v, scale = q.abs(), k.abs(), v.abs(), abs(scale)
        state = None if state is None else state.abs()
    B, (N, H, dk), dv = len(starts) - 1, q.shape, v.shape[2]
    o = torch.zeros(N, H, dv, dtype=torch.float64)
    last = torch.zeros(B, H, dk, dv, dtype=torch.float64)
    for b in range(B):
        S = torch.zeros(H, dk, dv, dtype=torch.float64) if state is None else f64(state)[b].clone()
        for t in range(starts[b], starts[b + 1]):
            S = lam[:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * torch.einsum("hd,hde->he", q[t], S)
        last[b] = S
    return o, last


def recurrence_grad(do, q, k, v, log_decay, scale, starts, state=None, dstate=None, magnitudes=False):
    """dq, dk, dv and the gradient of the first states."""
    do, q, k, v, lam = f64(do), f64(q), f64(k), f64(v), torch.exp(f64(log_decay))[:, None, None]
    if magnitudes:
        do, q, k, v, scale = do.abs(), q.abs(), k.abs(), v.abs(), abs(scale)
        state = None if state is None else state.abs()
        dstate = None if dstate is None else dstate.abs()
    B, (N, H, dk), dv = len(starts) - 1, q.shape, v.shape[2]
    dq, gk, gv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    first = torch.zeros(B, H, dk, dv, dtype=torch.float64)
    for b in range(B):
        S = torch.zeros(H, dk, dv, dtype=torch.float64) if state is None else f64(state)[b].clone()
        for t in range(starts[b], starts[b + 1]):
            S = lam * S + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * torch.einsum("hde,he->hd", S, do[t])
        G = torch.zeros(H, dk, dv, dtype=torch.float64) if dstate is None else f64(dstate)[b].clone()
        for t in range(starts[b + 1] - 1, starts[b] - 1, -1):
            G = G + scale * q[t][:, :, None] * do[t][:, None, :]
            gk[t] = torch.einsum("hde,he->hd", G, v[t])
            gv[t] = torch.einsum("hd,hde->he", k[t], G)
            G = lam * G
        first[b] = G
    return dq, gk, gv, first
