"""Timed cases of the gated feed-forward sublayer: the block in bf16 and fp32, its gradient, the encoding of
matrices in FP8 blocks of 128, the product of two such matrices, and the block on FP8 weights.

``run`` computes a case in plain torch operations in 32 bits (``own`` false) or through the library's public
calls (``own`` true) on what ``prepare`` made; ``exact`` gives the same outputs in 64 bits from the definition."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 128


def listed():
    return [
        # a decode step of a single request: nothing but the weights to read; latency counts
        {"name": "ff step", "op": "ff", "n": 1, "d": 2560, "f": 10240, "act": "silu", "dtype": "bf16", "keep": False},
        # a decode step of a batch of 64
        {"name": "ff decode", "op": "ff", "n": 64, "d": 4096, "f": 16384, "act": "silu", "dtype": "bf16",
         "keep": False},
        # the prompt batch of the prefill workload, 4 x 4096 tokens
        {"name": "ff prompt", "op": "ff", "n": 16384, "d": 4096, "f": 11008, "act": "silu", "dtype": "bf16",
         "keep": False},
        # fp32 states stand for small models and checks; a training step's forward pass, odd sizes
        {"name": "ff f32", "op": "ff", "n": 301, "d": 1000, "f": 2728, "act": "gelu", "dtype": "f32", "keep": True},
        # the block's gradients in a training step
        {"name": "ff grad", "op": "ff_grad", "n": 8192, "d": 2560, "f": 10240, "act": "silu", "dtype": "bf16"},
        # a small model's, sizes off every tile
        {"name": "ff grad small", "op": "ff_grad", "n": 509, "d": 1032, "f": 2744, "act": "gelu", "dtype": "bf16"},
        # a decode step's activations before a product
        {"name": "encode decode", "op": "encode", "n": 128, "k": 4096, "rows": 1, "dtype": "bf16"},
        # weights as a program lays them out once, from their fp32 master, a width that ends inside a block
        {"name": "encode weights", "op": "encode", "n": 16384, "k": 7184, "rows": 128, "dtype": "f32"},
        # a projection in a decode step of a batch of 64
        {"name": "product decode", "op": "product", "n": 64, "k": 4096, "o": 16384},
        # a projection of a packed prompt batch with an odd number of tokens
        {"name": "product prompt", "op": "product", "n": 8191, "k": 7168, "o": 4096},
        # a decode step of the block on FP8 weights
        {"name": "ff fp8 decode", "op": "ff_fp8", "n": 64, "d": 4096, "f": 16384, "act": "silu"},
        # the prefill workload's prompt batch on FP8 weights
        {"name": "ff fp8 prompt", "op": "ff_fp8", "n": 16384, "d": 4096, "f": 11008, "act": "silu"},
    ]


def _spread(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["ff", "ff", "ff_grad", "encode", "product", "ff_fp8"])
    n = _spread(rng, 1, 16384)
    if op == "encode":
        return {"op": op, "n": n, "k": 16 * _spread(rng, 4, 449), "rows": rng.choice([1, 1, 128]),
                "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "product":
        return {"op": op, "n": n, "k": 16 * _spread(rng, 8, 448), "o": 8 * _spread(rng, 16, 1376)}
    act = rng.choice(["silu", "silu", "gelu"])
    if op == "ff_fp8":
        return {"op": op, "n": n, "d": 16 * _spread(rng, 8, 256), "f": 16 * _spread(rng, 16, 688), "act": act}
    f32 = rng.random() < 0.2
    case = {"op": op, "n": _spread(rng, 1, 1024 if f32 else 16384 if op == "ff" else 8192),
            "d": 8 * _spread(rng, 16, 512 if op == "ff" else 320),
            "f": 8 * _spread(rng, 32, 1376 if op == "ff" else 1280), "act": act, "dtype": "f32" if f32 else "bf16"}
    if op == "ff":
        case.update(keep=rng.choice([True, False]))
    return case


# ---- inputs -------------------------------------------------------------------------------------

def _blocks(m, rows):
    """m [R, K] in 32 bits as [R/rows, rows, K/128, 128], zeros behind its ends."""
    r, k = m.shape
    m = torch.nn.functional.pad(m.float(), (0, -k % BLOCK, 0, -r % rows))
    return m.reshape(m.shape[0] // rows, rows, m.shape[1] // BLOCK, BLOCK)


def _encode(m, rows):
    """(e4m3 codes like m, biased exponents) of the blocks of rows x 128 values: the smallest power of two 2^e with
    the block's largest magnitude at most 448 * 2^e, e at least -127, which an all-zero block has."""
    b = _blocks(m, rows)
    part, power = torch.frexp(b.abs().amax((1, 3)))       # 448 = 0.875 * 2^9
    e = torch.where(part > 0, power - 9 + (part > 0.875).int(), -127).clamp(-127, 127)
    codes = (b * torch.exp2(-e.float())[:, None, :, None]).to(torch.float8_e4m3fn)
    codes = codes.view(torch.uint8).flatten(2).flatten(0, 1)[:m.shape[0], :m.shape[1]].contiguous()
    return codes, (e + 127).to(torch.uint8)


def _decode(codes, scales, rows):
    """The values in 32 bits."""
    e = torch.exp2(scales.float() - 127)
    e = e.repeat_interleave(rows, 0)[:codes.shape[0]].repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]
    return codes.view(torch.float8_e4m3fn).float() * e


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * std

    def rows(n, d):
        # reads of the residual: tokens of different size, one channel in a hundred far above the others
        x = normal(n, d) * torch.exp(0.5 * normal(n, 1))
        return x * torch.where(torch.rand(d, generator=gen, device="cuda") < 0.01, 20.0, 1.0)

    op, state = case["op"], dict(case=case)
    if op == "encode":
        m = rows(case["n"], case["k"]) if case["rows"] == 1 else normal(case["n"], case["k"], std=case["k"] ** -0.5)
        state.update(m=m.to(DTYPES[case["dtype"]]))
        return state
    if op == "product":
        n, k, o = case["n"], case["k"], case["o"]
        state.update(a=_encode(rows(n, k), 1), b=_encode(normal(o, k, std=k ** -0.5), BLOCK))
        return state
    n, d, f = case["n"], case["d"], case["f"]
    if op == "ff_fp8":
        gate, up = (_encode(normal(f, d, std=d ** -0.5), BLOCK) for _ in range(2))
        # the gate's and the up projection's weights, each with blocks of its own, in one buffer as a layer has them
        state.update(x=rows(n, d).bfloat16(), w_in=tuple(torch.stack(pair) for pair in zip(gate, up)),
                     w_out=_encode(normal(d, f, std=f ** -0.5), BLOCK))
        return state
    dtype = DTYPES[case["dtype"]]
    state.update(x=normal(n, d).to(dtype), w_in=normal(2, f, d, std=d ** -0.5).to(dtype),
                 w_out=normal(d, f, std=f ** -0.5).to(dtype))
    if op == "ff_grad":
        # the pre-activations as the forward pass left them
        state.update(dy=normal(n, d).to(dtype), pre=(state["x"] @ state["w_in"].flatten(0, 1).T).view(n, 2, f))
    return state


# ---- the plain forms ----------------------------------------------------------------------------

def _act(g, act):
    return g / (1 + torch.exp(-g)) if act == "silu" else 0.5 * g * (1 + torch.erf(g * 0.5 ** 0.5))


def _slope(g, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    return 0.5 * (1 + torch.erf(g * 0.5 ** 0.5)) + g * torch.exp(-0.5 * g * g) * (2 * math.pi) ** -0.5


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "encode":
        codes, scales = _encode(s["m"], case["rows"])
        return codes.view(torch.float8_e4m3fn), scales
    if op == "product":
        return (_decode(*s["a"], 1) @ _decode(*s["b"], BLOCK).T).bfloat16()
    n, f, act = case["n"], case["f"], case["act"]
    if op == "ff_fp8":
        x = _decode(*_encode(s["x"], 1), 1)
        gate, up = (x @ _decode(codes, scales, BLOCK).T for codes, scales in zip(*s["w_in"]))
        h = _decode(*_encode(_act(gate, act) * up, 1), 1)
        return (h @ _decode(*s["w_out"], BLOCK).T).bfloat16()
    x, w_in, w_out, dtype = s["x"].float(), s["w_in"].float().flatten(0, 1), s["w_out"].float(), s["x"].dtype
    if op == "ff":
        pre = (x @ w_in.T).view(n, 2, f)
        y = (_act(pre[:, 0], act) * pre[:, 1]) @ w_out.T
        return (y.to(dtype), pre.to(dtype)) if case["keep"] else y.to(dtype)
    dy, (gate, up) = s["dy"].float(), s["pre"].float().unbind(1)
    dh = dy @ w_out
    dpre = torch.stack([dh * up * _slope(gate, act), dh * _act(gate, act)], 1).flatten(1)
    dx, dw_in, dw_out = dpre @ w_in, dpre.T @ x, dy.T @ (_act(gate, act) * up)
    return dx.to(dtype), dw_in.view(2, f, case["d"]).to(dtype), dw_out.to(dtype)


def _library(s):
    from stream_gated_residual_gb300 import gr
    case = s["case"]
    op = case["op"]
    if op == "encode":
        codes, scales = gr.fp8_encode_blocks(s["m"], case["rows"])
        return codes.view(torch.float8_e4m3fn), scales
    if op == "product":
        return gr.fp8_matmul(s["a"], s["b"])
    if op == "ff_fp8":
        return gr.feed_forward_fp8(s["x"], s["w_in"], s["w_out"], case["act"])
    if op == "ff":
        return gr.feed_forward(s["x"], s["w_in"], s["w_out"], case["act"], keep=case["keep"])
    return gr.feed_forward_backward(s["dy"], s["x"], s["w_in"], s["w_out"], s["pre"], case["act"])


def run(state):
    return _library(state) if own else _plain(state)


def work(case):
    op, n = case["op"], case["n"]
    size = {"bf16": 2, "f32": 4}
    if op == "encode":
        k, blocks = case["k"], -(-n // case["rows"]) * -(-case["k"] // BLOCK)
        return {"bytes": n * k * (size[case["dtype"]] + 1) + blocks, "flops": 2 * n * k}
    if op == "product":
        k, o = case["k"], case["o"]
        kb = -(-k // BLOCK)
        return {"bytes": (n + o) * k + (n + -(-o // BLOCK)) * kb + 2 * n * o, "flops": 2 * n * k * o}
    d, f = case["d"], case["f"]
    if op == "ff_fp8":
        scales = 3 * -(-d // BLOCK) * -(-f // BLOCK)
        return {"bytes": 4 * n * d + 3 * d * f + scales, "flops": 6 * n * d * f}
    w = size[case["dtype"]]
    if op == "ff":
        return {"bytes": (2 * n * d + 3 * d * f + (2 * n * f if case["keep"] else 0)) * w, "flops": 6 * n * d * f}
    return {"bytes": (3 * n * d + 6 * d * f + 2 * n * f) * w, "flops": 12 * n * d * f}


# ---- the definitions in 64 bits -----------------------------------------------------------------

def _exact_codes(m, rows):
    """(values of the codes, exponents) of m in blocks, each rounded on e4m3's own grid: steps of 2^(q - 3) between
    2^q and 2^(q + 1), q at least -6, ties to even."""
    r, k = m.shape
    big = m.new_zeros(-(-r // rows) * rows, -(-k // BLOCK) * BLOCK)
    big[:r, :k] = m
    top = big.view(-1, rows, big.shape[1] // BLOCK, BLOCK).abs().amax((1, 3))
    e = torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -200)))
    # log2 may be off by a little next to a power of two
    e = torch.where(top > 448 * torch.exp2(e), e + 1, torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e))
    e = e.clamp(-127, 127)
    v = m / torch.exp2(e).repeat_interleave(rows, 0)[:r].repeat_interleave(BLOCK, 1)[:, :k]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step, e


def _exact_values(m, rows):
    codes, e = _exact_codes(m, rows)
    return codes * torch.exp2(e).repeat_interleave(rows, 0)[:m.shape[0]].repeat_interleave(BLOCK, 1)[:, :m.shape[1]]


def _of_codes(codes, scales, rows):
    """The values that given codes stand for, by e4m3's fields: sign, 4 bits of exponent, 3 of fraction."""
    c = codes.long()
    field, part = c >> 3 & 15, (c & 7).double()
    mag = torch.where(field > 0, (1 + part / 8) * torch.exp2(field.double() - 7), part / 8 * 2.0 ** -6)
    e = torch.exp2(scales.double() - 127)
    index = torch.arange(codes.shape[0], device=c.device)[:, None] // rows
    return torch.where(c >= 128, -mag, mag) * e[index, torch.arange(codes.shape[1], device=c.device) // BLOCK]


def _exact_act(g, act):
    """(the activation, its slope)"""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    below = 0.5 * torch.erfc(-g / math.sqrt(2))
    return g * below, below + g * torch.exp(-g.square() / 2) / math.sqrt(2 * math.pi)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "encode":
        codes, e = _exact_codes(s["m"].double(), case["rows"])
        return codes, (e + 127).to(torch.uint8)
    if op == "product":
        return torch.einsum("nk,ok->no", _of_codes(*s["a"], 1), _of_codes(*s["b"], BLOCK))
    act = case["act"]
    if op == "ff_fp8":
        x = _exact_values(s["x"].double(), 1)
        (g, u), (gs, us) = s["w_in"]
        h = _exact_act(torch.einsum("nd,fd->nf", x, _of_codes(g, gs, BLOCK)), act)[0]
        h *= torch.einsum("nd,fd->nf", x, _of_codes(u, us, BLOCK))
        return torch.einsum("nf,df->nd", _exact_values(h, 1), _of_codes(*s["w_out"], BLOCK))
    x, w_in, w_out = (s[k].double() for k in ("x", "w_in", "w_out"))
    if op == "ff":
        pre = torch.einsum("nd,pfd->npf", x, w_in)
        y = torch.einsum("nf,df->nd", _exact_act(pre[:, 0], act)[0] * pre[:, 1], w_out)
        return (y, pre) if case["keep"] else y
    dy, gate, up = s["dy"].double(), s["pre"][:, 0].double(), s["pre"][:, 1].double()
    a, slope = _exact_act(gate, act)
    dh = torch.einsum("nd,df->nf", dy, w_out)
    dpre = torch.stack([slope * up * dh, a * dh], 1)
    return torch.einsum("npf,pfd->nd", dpre, w_in), torch.einsum("npf,nd->pfd", dpre, x), \
        torch.einsum("nd,nf->df", dy, a * up)
