"""Timed cases of the decoder operators around the Gated Residual: the token embedding into the widened state
and its gradient, layer norm and its gradient, and linear attention with a decay for each head over prompts,
single tokens and backwards.

``run`` computes a case in plain torch operations in 32 bits (``own`` false) or through the library's public
calls (``own`` true) on what ``prepare`` made; ``exact`` gives the same outputs in 64 bits from the definition."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # one decode step of a batch of 64: an id per request into the four branches; latency counts
        {"name": "embed decode", "op": "embed", "n": 64, "d": 4096, "vocab": 65536, "branches": 4,
         "table": "bf16", "dtype": "bf16", "ids": "uniform"},
        # the prompt batch of the prefill workload, 4 x 4096 tokens, from an fp32 master table
        {"name": "embed prompt", "op": "embed", "n": 16384, "d": 4096, "vocab": 65536, "branches": 4,
         "table": "f32", "dtype": "bf16", "ids": "zipf"},
        # a training batch whose token counts follow Zipf's law: the commonest token has about a tenth of the rows
        {"name": "embed grad", "op": "embed_grad", "n": 16384, "d": 2560, "vocab": 32768, "branches": 4,
         "ids": "zipf"},
        # an odd small batch on a plain stream
        {"name": "embed grad small", "op": "embed_grad", "n": 777, "d": 1000, "vocab": 5003, "branches": 1,
         "ids": "uniform"},
        # the norm before the logits of a decode step
        {"name": "norm decode", "op": "norm", "n": 128, "d": 4096, "groups": 1, "dtype": "bf16", "bias": True},
        # the norm of every branch of a deep-stack state, odd number of tokens
        {"name": "norm branches", "op": "norm", "n": 8191, "d": 2048, "groups": 4, "dtype": "bf16", "bias": True},
        # the end of the stack in a training step
        {"name": "norm grad", "op": "norm_grad", "n": 16384, "d": 4096, "groups": 1, "dtype": "bf16",
         "bias": True},
        # fp32 states, a width off the powers of two, no bias
        {"name": "norm grad f32 branches", "op": "norm_grad", "n": 501, "d": 2568, "groups": 4, "dtype": "f32",
         "bias": False},
        # one long prompt, 32 heads of 128, going on from a cached state
        {"name": "mixer prompt", "op": "mixer", "lengths": "one", "n": 32768, "seqs": 1, "heads": 32, "dk": 128,
         "dv": 128, "dtype": "bf16", "state": True},
        # 24 prompts of very different lengths in one batch, heads of 64
        {"name": "mixer packed", "op": "mixer", "lengths": "ragged", "n": 9001, "seqs": 24, "heads": 16, "dk": 64,
         "dv": 64, "dtype": "bf16", "state": False},
        # a decode step: 64 requests, 32 heads, the states are what is read and written
        {"name": "mixer step", "op": "mixer_step", "n": 64, "heads": 32, "dk": 128, "dv": 128, "dtype": "bf16"},
        # the mixer's gradients in a training step, two sequences
        {"name": "mixer grad", "op": "mixer_grad", "lengths": "even", "n": 8192, "seqs": 2, "heads": 16,
         "dk": 128, "dv": 128, "dtype": "bf16", "state": False},
    ]


def _spread(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "mixer", "mixer_step", "mixer_grad"])
    if op in ("embed", "embed_grad"):
        d, nb = 8 * _spread(rng, 32, 512), rng.choice([1, 4])
        case = {"op": op, "n": _spread(rng, 1, 16384), "d": d, "vocab": _spread(rng, 1000, 32768), "branches": nb,
                "ids": rng.choice(["uniform", "zipf"])}
        if op == "embed":
            case.update(table=rng.choice(["bf16", "f32"]), dtype=rng.choice(["bf16", "bf16", "f32"]))
        return case
    if op in ("norm", "norm_grad"):
        g = rng.choice([1, 4])
        return {"op": op, "n": _spread(rng, 1, 16384 // g), "d": 8 * _spread(rng, 16, 512), "groups": g,
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "bias": rng.choice([True, False])}
    if op == "mixer_step":
        return {"op": op, "n": _spread(rng, 1, 64), "heads": _spread(rng, 1, 32), "dk": rng.choice([64, 128]),
                "dv": rng.choice([64, 128]), "dtype": rng.choice(["bf16", "bf16", "f32"])}
    f32 = rng.random() < 0.2  # fp32 states stand for small models and checks
    n = _spread(rng, 1, 2048 if f32 else 16384 if op == "mixer" else 8192)
    lengths = rng.choice(["one", "even", "ragged"])
    d = rng.choice([64, 128])
    return {"op": op, "lengths": lengths, "n": n, "seqs": 1 if lengths == "one" else min(n, _spread(rng, 2, 32)),
            "heads": _spread(rng, 1, 8 if f32 else 16), "dk": d, "dv": d, "dtype": "f32" if f32 else "bf16",
            "state": rng.choice([True, False])}


def _lengths(case):
    """The sequences' lengths: one, equal ones, or ones that fall off as 1/(i + 1), at least one token each."""
    n, b = case["n"], case["seqs"]
    if case["lengths"] == "ragged":
        total = sum(1.0 / (i + 1) for i in range(b))
        got = [1 + int((n - b) / (i + 1) / total) for i in range(b)]
    else:
        got = [n // b] * b
    got[b // 2] += n - sum(got)
    return got


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    state = dict(case=case)
    op = case["op"]
    if op in ("embed", "embed_grad"):
        n, d, vocab, nb = case["n"], case["d"], case["vocab"], case["branches"]
        u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
        # Zipf's law by the inverse of its continuous distribution: a rank r has about 1/(r ln V) of the tokens
        ids = (vocab ** u if case["ids"] == "zipf" else u * vocab).long().clamp_(0, vocab - 1)
        state.update(ids=(ids * 7919) % vocab if math.gcd(7919, vocab) == 1 else ids, scale=math.sqrt(d))
        rows = (n, d) if nb == 1 else (n, nb, d)
        if op == "embed":
            state.update(table=normal(vocab, d, dtype=DTYPES[case["table"]]).mul_(0.02))
        else:
            state.update(grad=normal(*rows))
    elif op in ("norm", "norm_grad"):
        n, d, g = case["n"], case["d"], case["groups"]
        rows, per = ((n, d), (d,)) if g == 1 else ((n, g, d), (g, d))
        x = normal(*rows) * torch.exp(normal(*rows[:-1], 1)) + 0.5 * normal(*rows[:-1], 1)
        state.update(x=x.to(DTYPES[case["dtype"]]), weight=1 + 0.2 * normal(*per),
                     bias=0.1 * normal(*per) if case["bias"] else None)
        if op == "norm_grad":
            xf = state["x"].float()
            mean = xf.mean(-1)
            state.update(grad=normal(*rows), mean=mean,
                         rstd=torch.rsqrt((xf - mean[..., None]).square().mean(-1) + EPS))
    else:
        n, h, dk, dv = case["n"], case["heads"], case["dk"], case["dv"]
        dtype = DTYPES[case["dtype"]]
        # views of one projection's output, as a model has them; keys of about unit length
        qkv = normal(n, h * (2 * dk + dv))
        qkv[:, h * dk:2 * h * dk] *= dk ** -0.5
        qkv = qkv.to(dtype)
        q, k, v = qkv.split([h * dk, h * dk, h * dv], dim=1)
        # the heads' memories reach from a few tokens to a thousand
        decay = -torch.exp2(-torch.linspace(1.0, 10.0, h, device="cuda"))
        state.update(q=q.unflatten(1, (h, dk)), k=k.unflatten(1, (h, dk)), v=v.unflatten(1, (h, dv)),
                     log_decay=decay, scale=dk ** -0.5)
        if op == "mixer_step":
            state.update(state=normal(n, h, dk, dv))
        else:
            lengths = _lengths(case)
            b, longest = len(lengths), max(lengths)
            starts = [0]
            for length in lengths:
                starts.append(starts[-1] + length)
            state.update(starts=torch.tensor(starts, dtype=torch.int32, device="cuda"), longest=longest,
                         state=normal(b, h, dk, dv) if case["state"] else None)
            if op == "mixer_grad":
                state.update(grad=normal(n, h, dv, dtype=dtype),
                             dstate=normal(b, h, dk, dv) if case["state"] else None)
    return state


# ---- the plain forms ----------------------------------------------------------------------------

CHUNK = 64


def _padded(x, s):
    """Packed rows [N, H, D] as [H, B, T, D] in 32 bits, zeros behind each sequence, T a multiple of CHUNK."""
    starts = s["starts"].long()
    t = torch.arange(-(-s["longest"] // CHUNK) * CHUNK, device=x.device)
    at = starts[:-1, None] + t
    inside = at < starts[1:, None]
    rows = x.float()[at.clamp(max=x.shape[0] - 1)] * inside[:, :, None, None]
    return rows.permute(2, 0, 1, 3)


def _packed(x, s, dtype):
    """The rows of [H, B, T, D] back in the packed order, rounded to dtype."""
    starts = s["starts"].long()
    row = torch.arange(int(s["case"]["n"]), device=x.device)
    seq = torch.searchsorted(starts, row, right=True) - 1
    return x.permute(1, 2, 0, 3)[seq, row - starts[seq]].to(dtype)


def _powers(log_decay, exponent):
    """exp(log_decay * exponent) [H, ...] where exponent >= 0, else 0."""
    g = log_decay.reshape(-1, *([1] * exponent.dim()))
    return torch.where(exponent >= 0, torch.exp(g * exponent.clamp(min=0)), 0.0)


def _mix(a, b, c, log_decay, first):
    """out_t = sum_{s <= t} decay^(t-s) (a_t . b_s) c_s + decay^(t+1) a_t first, by chunks; a, b [H, B, T, Da]."""
    h, nb, t, da = a.shape
    dc, nc = c.shape[-1], t // CHUNK
    a, b, c = (x.reshape(h, nb, nc, CHUNK, x.shape[-1]) for x in (a, b, c))
    i = torch.arange(CHUNK, device=a.device, dtype=torch.float32)
    scores = (a @ b.transpose(-1, -2)) * _powers(log_decay, i[:, None] - i[None, :])[:, None, None]
    out = scores @ c
    own_sum = (b * _powers(log_decay, CHUNK - 1 - i)[:, None, None, :, None]).transpose(-1, -2) @ c
    j = torch.arange(nc, device=a.device, dtype=torch.float32)
    between = _powers(log_decay, (j[:, None] - j[None, :] - 1) * CHUNK)
    begin = (between[:, None] @ own_sum.reshape(h, nb, nc, da * dc)).reshape(h, nb, nc, da, dc)
    if first is not None:
        begin = begin + _powers(log_decay, j * CHUNK)[:, None, :, None, None] * first[:, :, None]
    out = out + _powers(log_decay, i + 1)[:, None, None, :, None] * (a @ begin)
    return out.reshape(h, nb, t, dc)


def _plain_mixer(s):
    q, k, v = (_padded(s[x], s) for x in "qkv")
    first = None if s["state"] is None else s["state"].transpose(0, 1)
    out = _mix(q, k, v, s["log_decay"], first) * s["scale"]
    length = (s["starts"][1:] - s["starts"][:-1]).float()
    left = length[:, None] - 1 - torch.arange(q.shape[2], device=q.device)
    last = (k * _powers(s["log_decay"], left)[..., None]).transpose(-1, -2) @ v
    if first is not None:
        last = last + _powers(s["log_decay"], length)[..., None, None] * first
    return _packed(out, s, s["q"].dtype), last.transpose(0, 1).contiguous()


def _plain_mixer_grad(s):
    q, k, v, g = (_padded(s[x], s) for x in ("q", "k", "v", "grad"))
    g = g * s["scale"]
    decay = s["log_decay"]
    first = None if s["state"] is None else s["state"].transpose(0, 1)
    dq = _mix(g, v, k, decay, None if first is None else first.transpose(-1, -2))
    q_, k_, v_, g_ = (x.flip(2) for x in (q, k, v, g))
    dk = _mix(v_, g_, q_, decay, None).flip(2)
    dv = _mix(k_, q_, g_, decay, None).flip(2)
    dfirst = None
    if first is not None:
        dlast = s["dstate"].transpose(0, 1)
        length = (s["starts"][1:] - s["starts"][:-1]).float()
        t = torch.arange(q.shape[2], device=q.device)
        left = _powers(decay, length[:, None] - 1 - t)[..., None]
        dk = dk + left * (v @ dlast.transpose(-1, -2))
        dv = dv + left * (k @ dlast)
        dfirst = (q * _powers(decay, t + 1.0)[:, None, :, None]).transpose(-1, -2) @ g
        dfirst = (dfirst + _powers(decay, length)[..., None, None] * dlast).transpose(0, 1).contiguous()
    out = [_packed(x, s, s["q"].dtype) for x in (dq, dk, dv)]
    return (*out, dfirst)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "embed":
        rows = (s["table"][s["ids"]].float() * s["scale"]).to(DTYPES[case["dtype"]])
        nb = case["branches"]
        return rows if nb == 1 else rows[:, None].expand(-1, nb, -1).contiguous()
    if op == "embed_grad":
        rows = s["grad"] if case["branches"] == 1 else s["grad"].sum(1)
        return torch.zeros(case["vocab"], case["d"], device="cuda").index_add_(0, s["ids"], rows * s["scale"])
    if op == "norm":
        x = s["x"].float()
        mean = x.mean(-1)
        centred = x - mean[..., None]
        rstd = torch.rsqrt(centred.square().mean(-1) + EPS)
        y = centred * rstd[..., None] * s["weight"]
        return (y if s["bias"] is None else y + s["bias"]).to(s["x"].dtype), mean, rstd
    if op == "norm_grad":
        xh = (s["x"].float() - s["mean"][..., None]) * s["rstd"][..., None]
        u = s["grad"] * s["weight"]
        dx = (u - u.mean(-1, keepdim=True) - xh * (u * xh).mean(-1, keepdim=True)) * s["rstd"][..., None]
        return dx, (s["grad"] * xh).sum(0), s["grad"].sum(0) if case["bias"] else None
    if op == "mixer":
        return _plain_mixer(s)
    if op == "mixer_grad":
        return _plain_mixer_grad(s)
    q, k, v = (s[x].float() for x in "qkv")
    s["state"].mul_(torch.exp(s["log_decay"])[:, None, None]).add_(k[..., :, None] * v[..., None, :])
    out = (q[..., None, :] @ s["state"])[..., 0, :] * s["scale"]
    return out.to(s["q"].dtype), s["state"]


def _library(s):
    from stream_gated_residual_gb300 import gr
    case = s["case"]
    op = case["op"]
    if op == "embed":
        return gr.embed(s["table"], s["ids"], s["scale"], branches=case["branches"], dtype=DTYPES[case["dtype"]])
    if op == "embed_grad":
        return gr.embed_backward(s["grad"], s["ids"], case["vocab"], s["scale"])
    if op == "norm":
        return gr.layer_norm(s["x"], s["weight"], s["bias"], EPS, stats=True)
    if op == "norm_grad":
        return gr.layer_norm_backward(s["grad"], s["x"], s["weight"], s["mean"], s["rstd"], bias=case["bias"])
    if op == "mixer":
        return gr.linear_attention(s["q"], s["k"], s["v"], s["log_decay"], s["scale"], seq_starts=s["starts"],
                                   state=s["state"])
    if op == "mixer_grad":
        return gr.linear_attention_backward(s["grad"], s["q"], s["k"], s["v"], s["log_decay"], s["scale"],
                                            seq_starts=s["starts"], state=s["state"], dstate=s["dstate"])
    return gr.linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["scale"]), s["state"]


def run(state):
    return _library(state) if own else _plain(state)


def work(case):
    op, n = case["op"], case["n"]
    size = {"bf16": 2, "f32": 4}
    if op in ("embed", "embed_grad"):
        d, nb, vocab = case["d"], case["branches"], case["vocab"]
        if op == "embed":
            # a row is read for each id, at most the whole table once
            read = min(n, vocab) * d * size[case["table"]]
            return {"bytes": n * 8 + read + n * nb * d * size[case["dtype"]], "flops": n * d}
        return {"bytes": n * 8 + n * nb * d * 4 + vocab * d * 4, "flops": n * nb * d}
    if op in ("norm", "norm_grad"):
        e, per = n * case["groups"] * case["d"], case["groups"] * case["d"] * 4 * (2 if case["bias"] else 1)
        stats = n * case["groups"] * 8
        if op == "norm":
            return {"bytes": 2 * e * size[case["dtype"]] + per + stats, "flops": 7 * e}
        return {"bytes": e * (size[case["dtype"]] + 8) + per + stats + case["groups"] * case["d"] * 4,
                "flops": 12 * e}
    h, dk, dv, w = case["heads"], case["dk"], case["dv"], size[case["dtype"]]
    if op == "mixer_step":
        return {"bytes": n * h * (2 * dk * dv * 4 + (2 * dk + 2 * dv) * w), "flops": 5 * n * h * dk * dv}
    states = case["seqs"] * h * dk * dv * 4
    if op == "mixer":
        # the recurrence itself: an update and a read of the state a token and head
        return {"bytes": n * h * (2 * dk + 2 * dv) * w + states * (2 if case["state"] else 1),
                "flops": 4 * n * h * dk * dv}
    return {"bytes": n * h * (4 * dk + 3 * dv) * w + (3 * states if case["state"] else 0),
            "flops": 10 * n * h * dk * dv}


def exact(case, seed):
    """The outputs from the definitions, in 64 bits: the recurrences token by token over all sequences and heads."""
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "embed":
        rows = torch.nn.functional.one_hot(s["ids"], case["vocab"]).to(f64) @ s["table"].to(f64) \
            if case["n"] * case["vocab"] < 1 << 22 else s["table"].to(f64).index_select(0, s["ids"])
        rows = rows * s["scale"]
        return rows if case["branches"] == 1 else torch.stack([rows] * case["branches"], 1)
    if op == "embed_grad":
        # differences of running sums over the rows in the order of their ids
        order = torch.argsort(s["ids"])
        rows = s["grad"].to(f64)
        rows = (rows if case["branches"] == 1 else rows.sum(1))[order] * s["scale"]
        total = torch.cat([torch.zeros(1, case["d"], dtype=f64, device="cuda"), rows.cumsum(0)])
        bounds = torch.searchsorted(s["ids"][order], torch.arange(case["vocab"] + 1, device="cuda"))
        return total[bounds[1:]] - total[bounds[:-1]]
    if op == "norm":
        x = s["x"].to(f64)
        mean = x.mean(-1)
        var = (x.square().mean(-1) - mean.square())
        rstd = 1 / (var + EPS).sqrt()
        y = (x - mean[..., None]) * rstd[..., None] * s["weight"].to(f64)
        return (y if s["bias"] is None else y + s["bias"].to(f64)), mean, rstd
    if op == "norm_grad":
        # by the definition with the given statistics
        dy, r = s["grad"].to(f64), s["rstd"].to(f64)[..., None]
        xh = (s["x"].to(f64) - s["mean"].to(f64)[..., None]) * r
        u = dy * s["weight"].to(f64)
        d = case["d"]
        dx = r * (u - u.sum(-1, keepdim=True) / d - xh * ((u * xh).sum(-1, keepdim=True) / d))
        return dx, torch.einsum("n...,n...->...", dy, xh), dy.sum(0) if case["bias"] else None
    q, k, v = (s[x].to(f64) for x in "qkv")
    lam = torch.exp(s["log_decay"].to(f64))[:, None, None]
    if op == "mixer_step":
        new = lam * s["state"].to(f64) + torch.einsum("bhd,bhe->bhde", k, v)
        return torch.einsum("bhd,bhde->bhe", q, new) * s["scale"], new
    lengths = _lengths(case)
    b, h, dk, dv = len(lengths), case["heads"], case["dk"], case["dv"]
    if max(lengths) > 40000 or max(lengths) * b * h * dk * dv > 4e11:
        return None
    starts = s["starts"].long()[:-1]
    # sequences from the longest to the shortest, so that those still running are the first ones
    by = sorted(range(b), key=lambda i: -lengths[i])
    order = torch.tensor(by, device="cuda")
    live = [sum(1 for length in lengths if length > t) for t in range(max(lengths))]
    first = s["state"].to(f64) if s["state"] is not None else torch.zeros(b, h, dk, dv, dtype=f64, device="cuda")
    S = first[order].clone()
    begin = starts[order]
    if op == "mixer":
        out = torch.empty(case["n"], h, dv, dtype=f64, device="cuda")
        for t in range(max(lengths)):
            m = live[t]
            row = begin[:m] + t
            S[:m] = lam * S[:m] + k[row][..., :, None] * v[row][..., None, :]
            out[row] = (q[row][..., None, :] @ S[:m])[..., 0, :]
        last = torch.empty_like(S)
        last[order] = S
        return out * s["scale"], last
    g = s["grad"].to(f64) * s["scale"]
    dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t in range(max(lengths)):
        m = live[t]
        row = begin[:m] + t
        S[:m] = lam * S[:m] + k[row][..., :, None] * v[row][..., None, :]
        dq[row] = (S[:m] @ g[row][..., :, None])[..., 0]
    G = torch.zeros(b, h, dk, dv, dtype=f64, device="cuda")
    if s["dstate"] is not None:
        G = s["dstate"].to(f64)[order] / lam  # its first decay below takes it to the last token
    for t in range(max(lengths) - 1, -1, -1):
        m = live[t]
        row = begin[:m] + t
        G[:m] = lam * G[:m] + q[row][..., :, None] * g[row][..., None, :]
        dk_[row] = (G[:m] @ v[row][..., :, None])[..., 0]
        dv_[row] = (k[row][..., None, :] @ G[:m])[..., 0, :]
    if s["dstate"] is None:
        return dq, dk_, dv_, None
    dfirst = torch.empty_like(G)
    dfirst[order] = lam * G
    return dq, dk_, dv_, dfirst
