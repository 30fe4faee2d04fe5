"""Plain 64-bit forms of the gated feed-forward sublayer and of FP8 blocks, from their definitions, each with a
bound on what the library's arithmetic may differ by, elementwise.

A sum of K products is fp32, in any order: each of its additions is off by at most a unit in the last place of a
partial sum, 2^-23 of the sum of magnitudes (a tensor core may cut off where others round), so (K + 4)·2^-23 of it
covers the sum and the steps around it. A rounding to the call's dtype is off by 2^-8 (bf16) or 2^-24 (fp32)."""
from __future__ import annotations

import math

import torch

BLOCK = 128
ULP = 2.0 ** -23
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def f64(t):
    return t.detach().double()


def act(g, name):
    """(f(g), f'(g))"""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    below = 0.5 * torch.special.erfc(-g * 0.5 ** 0.5)
    return g * below, below + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def act_err(g):
    """What f(g) and f'(g) may be off by in fp32 given g: exp's relative error grows with its argument, by at most
    (4 + 2|g|) units; 1 + erf is off by a few units of 1; each is multiplied by g at most twice."""
    return (4 + 2 * g.abs()) * (1 + g.abs()) * ULP


SLOPE = 1.13      # the largest |f'| of either activation
CURVE = 0.8       # and of |f''|: 0.5 (silu), 0.798 (gelu)


def sums(a, b, K):
    """The error of fp32 sums over K of a[m, k] b[n, k]."""
    return (K + 4) * ULP * (a.abs() @ b.abs().T)


def forward(x, w_in, w_out, name, dtype):
    """y, pre and their bounds."""
    x, w_in, w_out, u = f64(x), f64(w_in), f64(w_out), ROUND[dtype]
    (N, D), F = x.shape, w_in.shape[1]
    gate, up = x @ w_in[0].T, x @ w_in[1].T
    eg, eu = sums(x, w_in[0], D), sums(x, w_in[1], D)
    a = act(gate, name)[0]
    h = a * up
    ea = SLOPE * eg + act_err(gate)
    eh = ea * up.abs() + a.abs() * eu + ea * eu
    eh = eh + u * (h.abs() + eh)
    y = h @ w_out.T
    ey = eh @ w_out.abs().T + sums(h.abs() + eh, w_out, F)
    pre, ep = torch.stack([gate, up], 1), torch.stack([eg, eu], 1)
    return y, pre, ey + u * (y.abs() + ey), ep + u * (pre.abs() + ep)


def backward(dy, x, w_in, w_out, pre, name, dtype):
    """[(gradient, bound)] of dx, dw_in, dw_out with the given pre."""
    dy, x, w_in, w_out, u = f64(dy), f64(x), f64(w_in), f64(w_out), ROUND[dtype]
    gate, up = f64(pre)[:, 0], f64(pre)[:, 1]
    (N, D), F = x.shape, w_out.shape[1]
    dh, edh = dy @ w_out, sums(dy, w_out.T, D)
    a, slope = act(gate, name)
    ea = act_err(gate)
    dg, du, h = dh * up * slope, dh * a, a * up
    edg = edh * (up * slope).abs() + (dh.abs() + edh) * up.abs() * ea
    edu = edh * a.abs() + (dh.abs() + edh) * ea
    edg, edu, eh = (e + u * (v.abs() + e) for e, v in ((edg, dg), (edu, du), (ea * up.abs(), h)))
    dpre, ep = torch.cat([dg, du], 1), torch.cat([edg, edu], 1)
    flat = w_in.flatten(0, 1)
    out = []
    for v, p, e, q, K in ((dpre @ flat, dpre, ep, flat.T, 2 * F), (dpre.T @ x, dpre.T, ep.T, x.T, N),
                          (h.T @ dy, h.T, eh.T, dy.T, N)):
        b = e @ q.abs().T + sums(p.abs() + e, q, K)
        out.append((v, b + u * (v.abs() + b)))
    dw_in, dw_out = out[1], out[2]
    return out[0], tuple(t.view(2, F, D) for t in dw_in), tuple(t.T for t in dw_out)


# ---- FP8 blocks ---------------------------------------------------------------------------------

def _tiled(v, m, rows):
    """v [.., R/rows, K/128] over the shape of m [.., R, K]."""
    return v.repeat_interleave(rows, -2)[..., :m.shape[-2], :].repeat_interleave(BLOCK, -1)[..., :m.shape[-1]]


def exponents(m, rows):
    """The smallest e with each block's largest magnitude at most 448·2^e, at least -127."""
    m = m.double().abs()
    m = torch.nn.functional.pad(m, (0, -m.shape[-1] % BLOCK, 0, -m.shape[-2] % rows))
    top = m.unflatten(-2, (-1, rows)).unflatten(-1, (-1, BLOCK)).amax((-3, -1))
    part, power = torch.frexp(top)          # 448 = 0.875 * 2^9
    e = torch.where(part > 0.875, power - 8, power - 9).double()
    return torch.where(top > 0, e, torch.full_like(e, -127)).clamp(-127, 127)


def on_grid(v):
    """v rounded to the e4m3 grid, ties to even: steps of 2^(q - 3) from 2^q on, q at least -6."""
    q = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(q - 3)
    return torch.round(v / step) * step


def encode(m, rows):
    """(codes' values, exponents)"""
    m, e = m.double(), exponents(m, rows)
    return on_grid(m / torch.exp2(_tiled(e, m, rows))), e


def decode(codes, scales, rows):
    c = codes.long()
    field, part = c >> 3 & 15, (c & 7).double()
    v = torch.where(field > 0, (1 + part / 8) * torch.exp2(field.double() - 7), part / 8 * 2.0 ** -6)
    v = torch.where(c >= 128, -v, v)
    v = torch.where((c & 127) == 127, torch.full_like(v, math.nan), v)
    e = torch.exp2(scales.double() - 127)
    return v * _tiled(torch.where(scales == 255, torch.full_like(e, math.nan), e), c, rows)


def product(a, b):
    """A Bᵀ of two matrices in blocks, and its bound."""
    a, b = decode(*a, 1), decode(*b, BLOCK)
    v, e = a @ b.T, sums(a, b, a.shape[1])
    return v, e + ROUND[torch.bfloat16] * (v.abs() + e)


def forward_fp8(x, w_in, w_out, name):
    """y and its bound: h's error may move a code to its neighbour, or a block that is next to a power of two to
    the next exponent."""
    codes, e = encode(x, 1)
    x = codes * torch.exp2(_tiled(e, codes, 1))
    w_in, w_out = decode(*w_in, BLOCK), decode(*w_out, BLOCK)
    (N, D), F = x.shape, w_in.shape[1]
    gate, up = x @ w_in[0].T, x @ w_in[1].T
    eg, eu = sums(x, w_in[0], D), sums(x, w_in[1], D)
    a = act(gate, name)[0]
    h = a * up
    ea = SLOPE * eg + act_err(gate)
    eh = ea * up.abs() + a.abs() * eu + ea * eu
    at, q, off = exponents(h, 1), None, torch.zeros_like(h)
    for shift in (0, -1, 1):
        e = torch.exp2(_tiled(at + shift, h, 1))
        code = [on_grid(v / e).clamp(-448, 448) * e for v in (h, h - eh, h + eh)]
        q = code[0] if shift == 0 else q
        wide = torch.maximum((code[1] - q).abs(), (code[2] - q).abs())
        if shift:      # only where h's error can move the block's largest magnitude across
            moved = (exponents(h.abs() + eh, 1) != at) | (exponents((h.abs() - eh).clamp(min=0), 1) != at)
            wide = torch.where(_tiled(moved, h, 1), torch.maximum(wide, (code[0] - q).abs()), 0.0)
        off = torch.maximum(off, wide)
    y = q @ w_out.T
    ey = off @ w_out.abs().T + sums(q.abs() + off, w_out, F)
    return y, ey + ROUND[torch.bfloat16] * (y.abs() + ey)
