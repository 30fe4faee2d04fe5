"""GPU parity of the decoder operators (embedding, layer norm, linear attention, their gradients)
against their 64-bit definitions. The bounds are the rounding errors of the arithmetic the header
states, elementwise: a sum of m fp32 products is within (m + c)·2^-24 of the sum of magnitudes, and
every rounding to bf16 within 2^-8 of what is rounded."""
from __future__ import annotations

import pytest
import torch

import decoder_ref as ref
from decoder_ref import U32, UBF, f64
from stream_gated_residual_gb300 import gr

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    gr.load()
    gr.device_status(clear=True)
    yield
    assert gr.device_status() == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def within(a, b, bound, what):
    over = ((f64(a) - b).abs() - bound).max().item() if b.numel() else -1.0
    assert over <= 0, f"{what}: {over:.3e} over the bound"


def rel(a, b):
    return ((f64(a) - b).norm() / b.norm().clamp(min=1e-300)).item()


# ---- embedding ----------------------------------------------------------------------------------

@pytest.mark.parametrize("table_dtype,dtype", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("N,V,D,nb,id_dtype", [(1, 1, 8, 4, torch.int64), (5, 17, 264, 1, torch.int32),
                                               (33, 100, 4096, 4, torch.int64), (700, 50, 1000, 4, torch.int32),
                                               (9, 3, 12288, 4, torch.int64)])
def test_embed(N, V, D, nb, id_dtype, table_dtype, dtype):
    g = gen(N + D)
    table = randn(g, V, D, dtype=table_dtype)
    ids = torch.randint(-2, V + 2, (N,), generator=g, device="cuda").to(id_dtype)
    R = gr.embed(table, ids, 1.7, branches=nb, dtype=dtype)
    ok = (ids >= 0) & (ids < V)
    rows = (table.float()[ids.long().clamp(0, V - 1)] * 1.7 * ok[:, None]).to(dtype)
    want = rows if nb == 1 else rows[:, None].expand(-1, 4, -1)
    assert R.dtype == dtype and torch.equal(R, want)


def test_embed_far_rows_and_unaligned_ids():
    """Rows past 2^31 elements of the table; ids that start off any 8-byte boundary."""
    V, D = 300_000, 8192
    table = torch.zeros(V, D, dtype=BF, device="cuda")
    table[-1] = 3.0
    ids = torch.tensor([0, V - 1, V, 1], dtype=torch.int32, device="cuda")[1:]
    R = gr.embed(table, ids, 0.5)
    assert R.shape == (3, 4, D) and (R[0] == 1.5).all() and (R[1:] == 0).all()


def ids_of(kind, N, V, g):
    if kind == "same":
        return torch.full((N,), V // 2, device="cuda")
    if kind == "distinct":
        return torch.randperm(V, generator=g, device="cuda")[:N]
    if kind == "outside":
        return torch.randint(-V, 0, (N,), generator=g, device="cuda")
    u = torch.rand(N, generator=g, device="cuda", dtype=torch.float64)
    return (V ** u).long() - 1 + torch.randint(0, 2, (N,), generator=g, device="cuda") * (V // 2)


@pytest.mark.parametrize("N,V,D,nb,kind", [
    (1, 1, 8, 4, "same"), (2, 5, 8, 1, "mixed"), (31, 7, 520, 4, "mixed"), (32, 40, 264, 1, "distinct"),
    (100, 255, 1000, 4, "outside"), (1000, 256, 512, 4, "mixed"), (1025, 257, 516 + 4, 1, "same"),
    (4097, 65535, 64, 1, "mixed"), (5000, 65536, 64, 4, "distinct"), (16384, 300, 72, 1, "mixed"),
    (16385, 70000, 24, 4, "mixed"), (40000, 11, 32, 1, "same"), (333, 20, 12288, 4, "mixed")])
def test_embed_backward(N, V, D, nb, kind):
    g = gen(N * 3 + V)
    ids = ids_of(kind, N, V, g)
    dR = randn(g, *((N, D) if nb == 1 else (N, nb, D)))
    dE = gr.embed_backward(dR, ids, V, 0.7)
    want, mags, count = ref.embed_grad(dR, ids, V, 0.7)
    within(dE, want, (count * nb + 4) * U32 * mags, "dE")
    assert torch.equal(dE, gr.embed_backward(dR, ids.int(), V, 0.7))      # the order is fixed
    before = randn(g, V, D)
    got = gr.embed_backward(dR, ids, V, 0.7, dtable=before.clone(), accumulate=True)
    tiles = -(-N // 16384)
    within(got, f64(before) + want, ((count * nb + 4 + tiles) * mags + (tiles + 1) * f64(before).abs()) * U32, "+=")


def test_embed_backward_without_tokens():
    dE = torch.full((10, 16), 5.0, device="cuda")
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    gr.embed_backward(torch.empty(0, 4, 16, device="cuda"), ids, 10, dtable=dE, accumulate=True)
    assert (dE == 5).all()
    gr.embed_backward(torch.empty(0, 4, 16, device="cuda"), ids, 10, dtable=dE)
    assert (dE == 0).all()


def test_embed_gradient_against_differences():
    """<dE, T> is the change of <R, dR> along T: the lookup is linear, so one difference is exact."""
    g = gen(5)
    N, V, D = 200, 30, 256
    table, T, dR = randn(g, V, D), randn(g, V, D), randn(g, N, 4, D)
    ids = torch.randint(0, V, (N,), generator=g, device="cuda")
    loss = lambda t: (gr.embed(t, ids, 1.5).double() * dR.double()).sum().item()  # noqa: E731
    change = (loss(table + T) - loss(table - T)) / 2
    slope = (gr.embed_backward(dR, ids, V, 1.5).double() * T.double()).sum().item()
    size = (gr.embed(T.abs() + table.abs(), ids, 1.5).double() * dR.double().abs()).sum().item()
    assert abs(change - slope) <= 4 * U32 * size


# ---- layer norm -----------------------------------------------------------------------------------

NORM = [(1, 8, 1), (3, 8, 4), (2, 24, 1), (5, 264, 4), (70, 512, 1), (37, 520, 4), (33, 1000, 1), (650, 2048, 4),
        (401, 4096, 1), (19, 4104, 4), (11, 8200, 1), (6, 12288, 4)]


def norm_inputs(N, D, G, dtype, offset=0.3):
    g = gen(N + D + G)
    rows, per = ((N, D), (D,)) if G == 1 else ((N, G, D), (G, D))
    x = (randn(g, *rows) * torch.exp(randn(g, *rows[:-1], 1)) + offset).to(dtype)
    return x, 1 + 0.3 * randn(g, *per), 0.2 * randn(g, *per), randn(g, *rows)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N,D,G", NORM)
def test_layer_norm(N, D, G, dtype):
    x, w, b, _ = norm_inputs(N, D, G, dtype)
    for bias in (b, None):
        y, mean, rstd = gr.layer_norm(x, w, bias, 1e-5, stats=True)
        y64, m64, r64, xh = ref.layer_norm(x, w, bias, 1e-5)
        # sums: 16 terms a thread, then at most ten levels of a tree; 64 covers the rest
        size = f64(x).abs().mean(-1)
        within(mean, m64, 64 * U32 * size, "mean")
        spread = (f64(x) - m64[..., None]).abs().mean(-1)
        within(rstd, r64, 64 * U32 * r64 * (1 + (size * r64) ** 2 * U32), "rstd")
        bound = 64 * U32 * (f64(w).abs() * r64[..., None] * (size[..., None] + f64(x).abs() + spread[..., None])
                            + y64.abs() + (0 if bias is None else f64(bias).abs()))
        within(y, y64, bound + (UBF * (y64.abs() + bound) if dtype == BF else 0), "y")
        assert torch.equal(gr.layer_norm(x, w, bias, 1e-5), y)
    z = x.clone()
    assert torch.equal(gr.layer_norm(z, w, b, 1e-5, y=z), gr.layer_norm(x, w, b, 1e-5))


def test_layer_norm_far_mean_and_constant_rows():
    """A mean a thousand times the spread keeps the variance; a constant row gives the bias."""
    x, w, b, _ = norm_inputs(16, 1024, 1, F32, offset=1000.0)
    y, _, r = gr.layer_norm(x, w, b, 1e-5, stats=True)
    y64, _, r64, _ = ref.layer_norm(x, w, b, 1e-5)
    within(y, y64, 64 * U32 * (f64(w).abs() * r64[:, None] * 2 * f64(x).abs() + y64.abs() + f64(b).abs()), "y")
    const = torch.full((4, 1024), 2.5, device="cuda", dtype=BF)
    assert torch.equal(gr.layer_norm(const, w, b), b.to(BF).expand(4, -1))


def test_layer_norm_rows_do_not_touch_each_other():
    x, w, b, dy = norm_inputs(40, 520, 4, F32)
    y = gr.layer_norm(x, w, b)
    bad = x.clone()
    bad[7, 2, 100], bad[9, 0, 0] = float("nan"), float("inf")
    z = gr.layer_norm(bad, w, b)
    keep = torch.ones(40, 4, dtype=torch.bool, device="cuda")
    keep[7, 2] = keep[9, 0] = False
    assert torch.equal(z[keep], y[keep]) and torch.isnan(z[7, 2]).all() and not torch.isfinite(z[9, 0]).any()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N,D,G", NORM + [(3001, 64, 1), (2003, 16, 4)])
def test_layer_norm_backward(N, D, G, dtype):
    x, w, b, dy = norm_inputs(N, D, G, dtype)
    _, mean, rstd = gr.layer_norm(x, w, b, 1e-5, stats=True)
    dx, dw, db = gr.layer_norm_backward(dy, x, w, mean, rstd)
    dx64, dw64, db64, size, wsize, bsize = ref.layer_norm_grad(dy, x, w, mean, rstd)
    within(dx, dx64, 64 * U32 * size, "dx")
    within(dw, dw64, (N + 64) * U32 * wsize, "dweight")
    within(db, db64, (N + 64) * U32 * bsize, "dbias")
    dx2, dw2, none = gr.layer_norm_backward(dy, x, w, mean, rstd, bias=False)
    assert none is None and torch.equal(dx2, dx) and torch.equal(dw2, dw)
    buf = dy.clone()
    assert torch.equal(gr.layer_norm_backward(buf, x, w, mean, rstd, dx=buf)[0], dx)


def test_layer_norm_gradient_against_differences():
    x, w, b, dy = norm_inputs(23, 520, 4, F32)
    _, mean, rstd = gr.layer_norm(x, w, b, 1e-5, stats=True)
    dx, dw, db = gr.layer_norm_backward(dy, x, w, mean, rstd)
    loss = lambda x, w, b: (gr.layer_norm(x, w, b, 1e-5).double() * dy.double()).sum().item()  # noqa: E731
    g = gen(3)
    for i, (t, grad) in enumerate(((x, dx), (w, dw), (b, db))):
        d = randn(g, *t.shape) * (t.std(-1, keepdim=True) if i == 0 else 1)
        h = 1e-2 if i == 0 else 0.5          # y is linear in w and b
        up, down = [x, w, b], [x, w, b]
        up[i], down[i] = t + h * d, t - h * d
        change = (loss(*up) - loss(*down)) / (2 * h)
        slope = (grad.double() * d.double()).sum().item()
        # truncation: h² of the third derivative, a few times the slope's own size; rounding: 64
        # roundoffs of every term of the two losses over h
        size = (grad.double() * d.double()).abs().sum().item()
        terms = (gr.layer_norm(x, w, b).double().abs() * dy.double().abs()).sum().item()
        assert abs(change - slope) <= (6 * h * h if i == 0 else 0) * size + 64 * U32 * terms / h


def test_layer_norm_backward_without_tokens():
    w = torch.ones(4, 64, device="cuda")
    x = torch.empty(0, 4, 64, device="cuda")
    st = torch.empty(0, 4, device="cuda")
    dx, dw, db = gr.layer_norm_backward(x, x, w, st, st)
    assert dx.shape == x.shape and (dw == 0).all() and (db == 0).all()


# ---- linear attention -----------------------------------------------------------------------------

def mixer_inputs(lengths, H, dk, dv, dtype, seed=0, layout="fused"):
    g = gen(seed + sum(lengths) + H + dk)
    N = sum(lengths)
    if layout == "fused":       # views of one projection's output
        qkv = randn(g, N, H * (2 * dk + dv), dtype=dtype)
        q, k, v = (t.unflatten(1, (H, -1)) for t in qkv.split([H * dk, H * dk, H * dv], 1))
    elif layout == "heads":     # head-major
        q, k, v = (randn(g, H, N, d, dtype=dtype).transpose(0, 1) for d in (dk, dk, dv))
    else:
        q, k, v = (randn(g, N, H, d, dtype=dtype) for d in (dk, dk, dv))
    starts = [0]
    for n in lengths:
        starts.append(starts[-1] + n)
    decay = -torch.exp2(-torch.linspace(0.0, 9.0, H, device="cuda"))
    state = randn(g, len(lengths), H, dk, dv)
    return q, k, v, decay, torch.tensor(starts, dtype=torch.int32, device="cuda"), starts, state, g


def mixer_bounds(out, mags, terms, dtype):
    """fp32 sums of `terms` products; on the bf16 path the output, the scores and the state are rounded."""
    return terms * U32 * mags + (UBF * (out.abs() + 1.01 * mags) if dtype == BF else 0)


MIX = [([1], 1, 8, 8), ([2], 3, 16, 24), ([31, 1, 0, 33], 2, 40, 72), ([0, 5], 1, 256, 256), ([64, 65], 2, 64, 64),
       ([127, 0, 129, 1], 2, 128, 128), ([300], 3, 64, 128), ([5, 257, 128], 2, 128, 64), ([200, 90], 1, 96, 200)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lengths,H,dk,dv", MIX)
def test_linear_attention(lengths, H, dk, dv, dtype):
    for layout, with_state in (("fused", True), ("heads", False)):
        q, k, v, decay, starts, at, state, _ = mixer_inputs(lengths, H, dk, dv, dtype, layout=layout)
        state = state if with_state else None
        o, last = gr.linear_attention(q, k, v, decay, 0.3, seq_starts=starts, state=state)
        o64, l64 = ref.recurrence(q, k, v, decay, 0.3, at, state)
        om, lm = ref.recurrence(q, k, v, decay, 0.3, at, state, magnitudes=True)
        terms = dk + 64 + 4 * (max(lengths) // 32 + 1)
        within(o, o64, mixer_bounds(o64, om, terms, dtype), "o")
        within(last, l64, (terms + 64) * U32 * lm, "state")
        if dtype == BF and o64.norm() > 0:
            assert rel(o, o64) <= 5e-3      # three roundings to bf16, 1.7e-3 each in the mean
        o2, last2 = gr.linear_attention(q, k, v, decay, 0.3, seq_starts=starts, state=state)
        assert torch.equal(o, o2) and torch.equal(last, last2)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_linear_attention_long(dtype):
    """A prompt long enough to be split over its length, heads that remember all of it."""
    q, k, v, decay, _, at, state, _ = mixer_inputs([5003], 2, 128, 128, dtype)
    decay = torch.tensor([-1e-4, 0.0], device="cuda")
    o, last = gr.linear_attention(q, k, v, decay, state=state)
    o64, l64 = ref.recurrence(q, k, v, decay, 128 ** -0.5, at, state)
    assert rel(o, o64) <= (5e-3 if dtype == BF else 1e-5)
    assert rel(last, l64) <= 2e-6


@pytest.mark.parametrize("dk,dv,dtype", [(128, 128, BF), (64, 128, BF), (128, 64, BF), (64, 64, F32), (96, 40, BF),
                                         (200, 72, F32)])
def test_linear_attention_cut_prompts(dk, dv, dtype):
    """Packed prompts that are cut into segments, forwards and backwards; the last states on top of the first."""
    tol = 5e-3 if dtype == BF else 1e-5
    lengths = [1500, 1, 0, 2100, 130]
    q, k, v, decay, starts, at, state, g = mixer_inputs(lengths, 2, dk, dv, dtype)
    decay = torch.tensor([-2e-3, -0.3], device="cuda")
    do, dstate = randn(g, *v.shape, dtype=dtype), randn(g, *state.shape)
    o, last = gr.linear_attention(q, k, v, decay, 0.3, seq_starts=starts, state=state)
    o64, l64 = ref.recurrence(q, k, v, decay, 0.3, at, state)
    assert rel(o, o64) <= tol and rel(last, l64) <= 2e-6
    onto = state.clone()
    o2, same = gr.linear_attention(q, k, v, decay, 0.3, seq_starts=starts, state=onto, state_out=onto)
    assert same is onto and torch.equal(o2, o) and torch.equal(onto, last)
    got = gr.linear_attention_backward(do, q, k, v, decay, 0.3, seq_starts=starts, state=state, dstate=dstate)
    want = ref.recurrence_grad(do, q, k, v, decay, 0.3, at, state, dstate)
    for a, b in zip(got[:3], want):
        assert rel(a, b) <= tol
    assert rel(got[3], want[3]) <= 2e-6


@pytest.mark.parametrize("dk,dv,dtype", [(128, 128, BF), (64, 64, BF), (64, 64, F32)])
def test_linear_attention_decays(dk, dv, dtype):
    """No decay, decays that underflow within a few tokens, and none of the past at all."""
    q, k, v, _, starts, at, state, _ = mixer_inputs([190, 130], 5, dk, dv, dtype)
    decay = torch.tensor([0.0, -float("inf"), -100.0, -20.0, -3e-3], device="cuda")
    o, last = gr.linear_attention(q, k, v, decay, 0.1, seq_starts=starts, state=state)
    o64, l64 = ref.recurrence(q, k, v, decay, 0.1, at, state)
    om, lm = ref.recurrence(q, k, v, decay, 0.1, at, state, magnitudes=True)
    within(o, o64, mixer_bounds(o64, om, dk + 100, dtype) + 1e-30, "o")
    within(last, l64, (dk + 164) * U32 * lm + 1e-30, "state")


@pytest.mark.parametrize("dk,dv,dtype", [(128, 128, BF), (64, 128, BF), (64, 64, F32)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_linear_attention_nothing_leaks(dk, dv, dtype, value):
    """What is not finite reaches neither an earlier token nor another sequence, whichever input has it."""
    lengths = [70, 150, 9, 40]
    q, k, v, decay, starts, at, state, _ = mixer_inputs(lengths, 2, dk, dv, dtype, layout="plain")
    o, last = gr.linear_attention(q, k, v, decay, seq_starts=starts, state=state)
    bad_token = at[1] + 101
    for name in ("q", "k", "v"):
        args = {"q": q.clone(), "k": k.clone(), "v": v.clone()}
        args[name][bad_token, 1, 5] = value
        z, zl = gr.linear_attention(args["q"], args["k"], args["v"], decay, seq_starts=starts, state=state)
        hit = torch.zeros(len(o), 2, dtype=torch.bool, device="cuda")
        hit[bad_token:(bad_token + 1 if name == "q" else at[2]), 1] = True
        assert torch.equal(z[~hit], o[~hit]), name
        assert not torch.isfinite(z[bad_token, 1]).all()
        keep = torch.ones(4, 2, dtype=torch.bool, device="cuda")
        keep[1, 1] = name == "q"
        assert torch.equal(zl[keep], last[keep]), name
    # rows that no sequence holds are not read into one and not written
    args = [t.clone() for t in (q, k, v)]
    for t in args:
        t[at[3]:] = value
    out = torch.full_like(o, 7.0)
    z, zl = gr.linear_attention(*args, decay, seq_starts=starts[:4].contiguous(), state=state[:3].contiguous(), o=out)
    assert torch.equal(z[:at[3]], o[:at[3]]) and (z[at[3]:] == 7).all() and torch.equal(zl, last[:3])


@pytest.mark.parametrize("lengths,H,dk,dv", [([129], 1, 128, 128), ([200, 1, 55], 1, 64, 64), ([300], 4, 64, 128),
                                             ([511, 257], 2, 128, 64), ([2048], 1, 128, 128)])
def test_linear_attention_few_rows_are_rounded_once(lengths, H, dk, dv):
    """Calls of few rows have the error of the output's rounding, forwards and in every gradient: the
    scores' and the state's two terms leave at most 2^-17 of them, less than 1/100 of that rounding."""
    q, k, v, decay, starts, at, state, g = mixer_inputs(lengths, H, dk, dv, BF)
    do, dstate = randn(g, *v.shape, dtype=BF), randn(g, *state.shape)
    o, _ = gr.linear_attention(q, k, v, decay, 0.3, seq_starts=starts, state=state)
    o64, _ = ref.recurrence(q, k, v, decay, 0.3, at, state)
    got = gr.linear_attention_backward(do, q, k, v, decay, 0.3, seq_starts=starts, state=state, dstate=dstate)
    want = ref.recurrence_grad(do, q, k, v, decay, 0.3, at, state, dstate)
    for a, b in ((o, o64), *zip(got[:3], want)):
        assert rel(a, b) <= 1.05 * rel(b.to(BF), b)


@pytest.mark.parametrize("lengths,H,dk,dv", [([127, 0, 129, 1], 9, 128, 128), ([300], 7, 64, 128), ([5, 257, 128], 6, 128, 64),
                                             ([700], 3, 64, 64)])
def test_linear_attention_more_rows(lengths, H, dk, dv):
    """Sizes above those that are rounded once: forwards, gradients, and what is not finite stays where it is."""
    q, k, v, decay, starts, at, state, g = mixer_inputs(lengths, H, dk, dv, BF, layout="plain")
    do, dstate = randn(g, *v.shape, dtype=BF), randn(g, *state.shape)
    o, last = gr.linear_attention(q, k, v, decay, 0.3, seq_starts=starts, state=state)
    o64, l64 = ref.recurrence(q, k, v, decay, 0.3, at, state)
    om, lm = ref.recurrence(q, k, v, decay, 0.3, at, state, magnitudes=True)
    terms = dk + 64 + 4 * (max(lengths) // 32 + 1)
    within(o, o64, mixer_bounds(o64, om, terms, BF), "o")
    within(last, l64, (terms + 64) * U32 * lm, "state")
    got = gr.linear_attention_backward(do, q, k, v, decay, 0.3, seq_starts=starts, state=state, dstate=dstate)
    want = ref.recurrence_grad(do, q, k, v, decay, 0.3, at, state, dstate)
    for a, b in zip(got[:3], want):
        assert rel(a, b) <= 5e-3
    assert rel(got[3], want[3]) <= 2e-6
    bad = 1 + lengths[0] // 2
    for value in (float("nan"), float("inf")):
        for name in ("q", "k", "v"):
            args = {"q": q.clone(), "k": k.clone(), "v": v.clone()}
            args[name][bad, 1, 5] = value
            z, zl = gr.linear_attention(args["q"], args["k"], args["v"], decay, 0.3, seq_starts=starts, state=state)
            hit = torch.zeros(len(o), H, dtype=torch.bool, device="cuda")
            hit[bad:(bad + 1 if name == "q" else at[1]), 1] = True
            assert torch.equal(z[~hit], o[~hit]), name
            assert not torch.isfinite(z[bad, 1]).all(), name


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 32)])
def test_linear_attention_split_prompt_and_steps(dtype, d):
    """A prompt in two parts through the state, and its last tokens one by one, give the whole one's."""
    q, k, v, decay, _, at, state, _ = mixer_inputs([260], 2, d, d, dtype)
    o, last = gr.linear_attention(q, k, v, decay, state=state)
    a, mid = gr.linear_attention(q[:141], k[:141], v[:141], decay, state=state)
    b, end = gr.linear_attention(q[141:250], k[141:250], v[141:250], decay, state=mid, state_out=mid)
    assert end is mid or end.data_ptr() == mid.data_ptr()
    rows = [gr.linear_attention_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], decay, end) for t in range(250, 260)]
    got = torch.cat([a, b, *rows])
    assert rel(got, f64(o)) <= (7e-3 if dtype == BF else 1e-5)
    assert rel(end, f64(last)) <= 4e-6


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N,H,dk,dv", [(1, 1, 8, 8), (3, 2, 40, 72), (17, 5, 64, 64), (5, 3, 256, 256), (64, 4, 128, 128),
                                       (2, 1, 128, 200)])
def test_linear_attention_step(N, H, dk, dv, dtype):
    q, k, v, decay, _, _, state, g = mixer_inputs([1] * N, H, dk, dv, dtype)
    pool = randn(g, N + 3, H, dk, dv)
    slots = torch.randperm(N + 3, generator=g, device="cuda")[:N].int()
    if N > 2:
        slots[1], slots[2] = -1, N + 3
    before = pool.clone()
    o = gr.linear_attention_step(q, k, v, decay, pool, 0.3, slots=slots)
    live = [i for i in range(N) if 0 <= slots[i] < N + 3]
    used = slots[live].long()
    starts = list(range(len(live) + 1))
    args = (q[live], k[live], v[live], decay, 0.3, starts, before[used])
    o64, l64 = ref.recurrence(*args)
    om, lm = ref.recurrence(*args, magnitudes=True)
    within(o[live], o64, (dk + 16) * U32 * om + (UBF * o64.abs() * 1.01 if dtype == BF else 0), "o")
    within(pool[used], l64, 4 * U32 * lm, "state")
    rest = torch.ones(N + 3, dtype=torch.bool, device="cuda")
    rest[used] = False
    assert torch.equal(pool[rest], before[rest])
    if N > 2:
        assert (o[1] == 0).all() and (o[2] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lengths,H,dk,dv", MIX)
def test_linear_attention_backward(lengths, H, dk, dv, dtype):
    for with_state in (True, False):
        q, k, v, decay, starts, at, state, g = mixer_inputs(lengths, H, dk, dv, dtype)
        do = randn(g, *v.shape, dtype=dtype)
        dstate = randn(g, *state.shape) if with_state else None
        state = state if with_state else None
        got = gr.linear_attention_backward(do, q, k, v, decay, 0.3, seq_starts=starts, state=state, dstate=dstate)
        want = ref.recurrence_grad(do, q, k, v, decay, 0.3, at, state, dstate)
        mags = ref.recurrence_grad(do, q, k, v, decay, 0.3, at, state, dstate, magnitudes=True)
        terms = max(dk, dv) + 64 + 4 * (max(lengths) // 32 + 1)
        for name, a, b, m in zip(("dq", "dk", "dv"), got, want, mags):
            within(a, b, mixer_bounds(b, m, terms, dtype), name)
            if dtype == BF and b.norm() > 0:
                assert rel(a, b) <= 5e-3
        if with_state:
            within(got[3], want[3], (terms + 64) * U32 * mags[3], "dstate")
        else:
            assert got[3] is None


def test_linear_attention_gradient_against_differences():
    """o and the last state are linear in each of q, k (through scores), v and the first state, so one
    central difference along a direction is exact but for rounding."""
    q, k, v, decay, starts, at, state, g = mixer_inputs([50, 33], 2, 64, 64, F32)
    do, ds = randn(g, *v.shape), randn(g, *state.shape)
    grads = gr.linear_attention_backward(do, q, k, v, decay, 0.2, seq_starts=starts, state=state, dstate=ds)

    def loss(args, absolute=False):
        if absolute:
            o, l = ref.recurrence(*args[:3], decay, 0.2, at, args[3], magnitudes=True)
            return ((o * f64(do).abs()).sum() + (l * f64(ds).abs()).sum()).item()
        o, l = gr.linear_attention(*args[:3], decay, 0.2, seq_starts=starts, state=args[3])
        return ((o.double() * do.double()).sum() + (l.double() * ds.double()).sum()).item()

    base = [q.contiguous(), k.contiguous(), v.contiguous(), state]
    for i in range(4):
        d = randn(g, *base[i].shape)
        up, down, both = list(base), list(base), list(base)
        up[i], down[i], both[i] = base[i] + d, base[i] - d, base[i].abs() + d.abs()
        change = (loss(up) - loss(down)) / 2
        slope = (grads[i].double() * d.double()).sum().item()
        assert abs(change - slope) <= 2 * (64 + 64 + 16) * U32 * loss(both, absolute=True)


def test_linear_attention_outputs_between_inputs():
    """Gradients written as views of one projection-shaped buffer, on another stream than the inputs'."""
    H, d = 3, 64
    q, k, v, decay, starts, at, _, g = mixer_inputs([100, 29], H, d, d, BF)
    do = randn(g, 129, H, d, dtype=BF)
    want = gr.linear_attention_backward(do, q, k, v, decay, seq_starts=starts)
    buf = torch.zeros(129, 3 * H * d + 64, dtype=BF, device="cuda")
    views = [buf[:, i * H * d:(i + 1) * H * d].unflatten(1, (H, d)) for i in range(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gr.linear_attention_backward(do, q, k, v, decay, seq_starts=starts, out=views, stream=side)
    side.synchronize()
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a, b)
    assert (buf[:, 3 * H * d:] == 0).all()


def test_operators_in_a_graph():
    """Captured once and replayed on new inputs: nothing is kept from the call that was captured."""
    g = gen(9)
    D, V, N, H, d = 256, 50, 40, 2, 64
    table, ids = randn(g, V, D), torch.randint(0, V, (N,), generator=g, device="cuda")
    w, b, decay = torch.ones(D, device="cuda"), torch.zeros(D, device="cuda"), torch.tensor([-0.1, -0.01], device="cuda")

    def step():
        x = gr.embed(table, ids, 2.0, branches=1, dtype=BF)
        y, mean, rstd = gr.layer_norm(x, w, b, stats=True)
        q, k, v = (y[:, i * 64:i * 64 + H * d].unflatten(1, (H, d)) for i in range(3))
        o, s = gr.linear_attention(q, k, v, decay)
        grads = gr.linear_attention_backward(o, q, k, v, decay)
        dx, dw, db = gr.layer_norm_backward(y.float(), x, w, mean, rstd)
        return [y, o, s, *grads[:3], dx, dw, db, gr.embed_backward(dx, ids, V)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (1, 2):
        table.copy_(randn(gen(seed), V, D))
        ids.copy_(torch.randint(0, V, (N,), generator=gen(seed), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(outs, step()):
            assert torch.equal(a, c)


@pytest.mark.parametrize("dtype,H,d", [(BF, 3, 64), (BF, 2, 128), (F32, 3, 24)])
def test_linear_attention_outputs_between_heads(dtype, H, d):
    """o between q, k and v of every head in one buffer [N, H, 4, d], and the gradients in one [N, H, 3, d]: the
    same bits as in buffers of their own, and nothing else is written."""
    q, k, v, decay, starts, at, _, g = mixer_inputs([100, 29, 140], H, d, d, dtype, layout="plain")
    N = len(q)
    do = randn(g, N, H, d, dtype=dtype)
    want, last = gr.linear_attention(q, k, v, decay, seq_starts=starts)
    grads = gr.linear_attention_backward(do, q, k, v, decay, seq_starts=starts)
    buf = torch.stack([q, k, v, torch.zeros_like(q)], 2)
    parts = buf.unbind(2)
    o, end = gr.linear_attention(*parts[:3], decay, seq_starts=starts, o=parts[3])
    assert torch.equal(o, want) and torch.equal(end, last)
    for a, b in zip(parts, (q, k, v)):
        assert torch.equal(a, b)
    out = torch.zeros(N, H, 3, d, dtype=dtype, device="cuda")
    got = gr.linear_attention_backward(do, *parts[:3], decay, seq_starts=starts, out=out.unbind(2))
    for a, b in zip(got[:3], grads[:3]):
        assert torch.equal(a, b)
    with pytest.raises(gr.GRError):
        gr.linear_attention(*parts[:3], decay, seq_starts=starts, o=parts[1])


def test_outputs_dropped_early_on_another_stream():
    """An output that the caller drops while its stream still runs is not handed out again before that."""
    g = gen(3)
    x, w = randn(g, 20000, 4, 1024), torch.ones(4, 1024, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gr.layer_norm(x, w)                                   # (the library and its kernel are loaded)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)                    # about 0.1 s: what follows on `side` is still to come
    y = gr.layer_norm(x, w, stream=side)
    at = y.data_ptr()
    del y
    other = torch.zeros_like(x)
    assert not side.query() and other.data_ptr() != at
    side.synchronize()
    assert (other == 0).all()


@pytest.mark.parametrize("lengths", [[5, 0, 130, 1], [1500, 1, 0, 2100, 130]])
@pytest.mark.parametrize("dk,dv,dtype", [(128, 128, BF), (64, 64, BF), (64, 128, BF), (64, 64, F32), (200, 72, F32)])
def test_linear_attention_state_gradient_in_place(lengths, dk, dv, dtype):
    """dstate_in in dstate's own buffer: the gradients of the definition. (dv then runs after dk by itself,
    cut by a plan of its own.)"""
    q, k, v, decay, starts, at, state, g = mixer_inputs(lengths, 2, dk, dv, dtype)
    decay = torch.tensor([-2e-3, -0.3], device="cuda")
    do, dstate = randn(g, *v.shape, dtype=dtype), randn(g, *state.shape)
    onto = dstate.clone()
    got = gr.linear_attention_backward(do, q, k, v, decay, 0.3, seq_starts=starts, state=state, dstate=onto,
                                       dstate_in=onto)
    assert got[3] is onto
    want = ref.recurrence_grad(do, q, k, v, decay, 0.3, at, state, dstate)
    for a, b in zip(got[:3], want):
        assert rel(a, b) <= (5e-3 if dtype == BF else 1e-5)
    assert rel(onto, want[3]) <= 2e-6
    mags = ref.recurrence_grad(do, q, k, v, decay, 0.3, at, state, dstate, magnitudes=True)
    terms = max(dk, dv) + 64 + 4 * (max(lengths) // 32 + 1)
    for a, b, m in zip(got[:3], want, mags):
        within(a, b, mixer_bounds(b, m, terms, dtype), "gradient")
    within(onto, want[3], (terms + 64) * U32 * mags[3], "dstate_in")


@pytest.mark.parametrize("N,V,D,nb", [(1, 3, 8, 1), (777, 50, 1000, 1), (2048, 9, 64, 4), (16384, 300, 520, 1),
                                      (16384 + 600, 400, 520, 1), (2 * 16384 + 6000, 100, 16, 4)])
def test_embed_backward_stays_in_its_workspace(N, V, D, nb):
    """A workspace of the size asked for, between guards: the same gradient, the guards untouched."""
    g = gen(N)
    ids = torch.randint(-1, V + 1, (N,), generator=g, device="cuda")
    dR = randn(g, N, D) if nb == 1 else randn(g, N, nb, D)
    e = gr._embed_desc(N, V, D, nb, gr.GR_F32, gr.GR_F32, 64, 0.5)
    need = gr._need("gr_embed_backward_workspace_size", e)
    assert need % 256 == 0
    buf = torch.full((need + 8192,), 0x5a, dtype=torch.uint8, device="cuda")
    got = gr.embed_backward(dR, ids, V, 0.5, workspace=buf[4096:4096 + need])
    assert (buf[:4096] == 0x5a).all() and (buf[4096 + need:] == 0x5a).all()
    g64, m64, rows = ref.embed_grad(dR, ids, V, 0.5)
    within(got, g64, (rows * nb + 8) * U32 * m64, "gradient")


# Prompts and gradients on the tensor cores come in variants: `fine` up to 128 tokens or 2048 rows (tokens ·
# heads), and above that with or without a state as a result. The tests below say which one they mean.

def above_few_rows(lengths, H):
    N = sum(lengths)
    assert N > 128 and N * H > 2048, "the sizes of the variant that rounds scores and states once"


def cut(N, B, H, dk, dv, dtype, gradient):
    """Whether a call of these sizes can be cut into segments: only then it needs a workspace."""
    m = gr._mixer_desc(N, B, H, dk, dv, gr._DTYPES[dtype], 1.0)
    return gr._need("gr_linear_attention_workspace_size", m, int(gradient)) > 0


NO_STATE = [([127, 0, 129, 1], 9, 128, 128), ([300], 7, 64, 128), ([5, 257, 128], 6, 128, 64), ([700], 3, 64, 64),
            ([1500, 1, 0, 2100, 130], 2, 128, 128), ([1500, 1, 0, 2100, 130], 2, 64, 64), ([2900, 300], 1, 64, 128),
            ([3000], 2, 128, 64)]


@pytest.mark.parametrize("lengths,H,dk,dv", NO_STATE)
def test_linear_attention_no_state_is_a_result(lengths, H, dk, dv):
    """Training's ordinary call: no state in or out. The decayed values are then two bf16 terms (2^-17 of them is
    cut off, less than 1/100 of the roundings that mixer_bounds() counts)."""
    above_few_rows(lengths, H)
    assert max(lengths) < 1000 or cut(sum(lengths), len(lengths), H, dk, dv, BF, True)
    q, k, v, _, starts, at, _, g = mixer_inputs(lengths, H, dk, dv, BF)
    decay = -torch.exp2(-torch.linspace(2.0, 9.0, H, device="cuda"))
    do = randn(g, *v.shape, dtype=BF)
    terms = max(dk, dv) + 64 + 4 * (max(lengths) // 32 + 1)
    got = gr.linear_attention_backward(do, q, k, v, decay, 0.3, seq_starts=starts)
    assert got[3] is None
    want = ref.recurrence_grad(do, q, k, v, decay, 0.3, at)
    mags = ref.recurrence_grad(do, q, k, v, decay, 0.3, at, magnitudes=True)
    for name, a, b, m in zip(("dq", "dk", "dv"), got, want, mags):
        within(a, b, mixer_bounds(b, m, terms, BF) + 2 ** -16 * m, name)
        assert rel(a, b) <= 5e-3, name
    # a prompt whose last states nobody asks for (the C entry's state_out NULL)
    N = len(q)
    o = torch.empty(N, H, dv, dtype=BF, device="cuda")
    m = gr._mixer_desc(N, len(lengths), H, dk, dv, gr.GR_BF16, 0.3)
    wp, wn, _keep = gr._ws(gr._need("gr_linear_attention_workspace_size", m, 0), None, q, None)
    gr._call("gr_linear_attention", m, gr._rows(q, "q", N, H, dk, BF), gr._rows(k, "k", N, H, dk, BF),
             gr._rows(v, "v", N, H, dv, BF), decay.data_ptr(), starts.data_ptr(), None, gr._rows(o, "o", N, H, dv, BF),
             None, wp, wn, gr._raw_stream(None, q))
    o64, _ = ref.recurrence(q, k, v, decay, 0.3, at)
    om, _ = ref.recurrence(q, k, v, decay, 0.3, at, magnitudes=True)
    within(o, o64, mixer_bounds(o64, om, terms, BF) + 2 ** -16 * om, "o")
    assert rel(o, o64) <= 5e-3


@pytest.mark.parametrize("with_state", [True, False])
@pytest.mark.parametrize("dk,dv,dtype", [(128, 128, BF), (64, 64, BF), (64, 128, BF), (64, 64, F32)])
def test_linear_attention_decays_of_many_rows(dk, dv, dtype, with_state):
    """No decay, decays that underflow within a few tokens, and none of the past at all, forwards and backwards, in
    more rows than are rounded once and in prompts that are cut."""
    lengths, H = [190, 1300, 130], 5
    above_few_rows(lengths, H)
    assert cut(sum(lengths), 3, H, dk, dv, dtype, False)
    q, k, v, _, starts, at, state, g = mixer_inputs(lengths, H, dk, dv, dtype)
    decay = torch.tensor([0.0, -float("inf"), -100.0, -20.0, -3e-3], device="cuda")
    do, dstate = randn(g, *v.shape, dtype=dtype), randn(g, *state.shape)
    if not with_state:
        state = dstate = None
    terms = max(dk, dv) + 64 + 4 * (max(lengths) // 32 + 1)
    o, last = gr.linear_attention(q, k, v, decay, 0.1, seq_starts=starts, state=state)
    o64, l64 = ref.recurrence(q, k, v, decay, 0.1, at, state)
    om, lm = ref.recurrence(q, k, v, decay, 0.1, at, state, magnitudes=True)
    within(o, o64, mixer_bounds(o64, om, terms, dtype) + 1e-30, "o")
    within(last, l64, (terms + 64) * U32 * lm + 1e-30, "state")
    got = gr.linear_attention_backward(do, q, k, v, decay, 0.1, seq_starts=starts, state=state, dstate=dstate)
    want = ref.recurrence_grad(do, q, k, v, decay, 0.1, at, state, dstate)
    mags = ref.recurrence_grad(do, q, k, v, decay, 0.1, at, state, dstate, magnitudes=True)
    for name, a, b, m in zip(("dq", "dk", "dv"), got, want, mags):
        within(a, b, mixer_bounds(b, m, terms, dtype) + (2 ** -16 * m if dtype == BF else 0) + 1e-30, name)
    if with_state:
        within(got[3], want[3], (terms + 64) * U32 * mags[3] + 1e-30, "dstate_in")


@pytest.mark.parametrize("dk,dv,dtype", [(64, 64, BF), (128, 64, BF), (32, 40, F32)])
def test_linear_attention_many_sequences(dk, dv, dtype):
    """More sequences than a warp has lanes, more (sequence, head) rows than SMs, and long ones behind the 32nd and the
    64th that are cut all the same."""
    g = gen(17)
    lengths = torch.randint(0, 25, (70,), generator=g, device="cuda").tolist()
    lengths[3], lengths[40], lengths[66] = 0, 5000, 3500
    H, N, tol = 4, sum(lengths), 5e-3 if dtype == BF else 1e-5
    assert len(lengths) * H >= 152
    assert cut(N, 70, H, dk, dv, dtype, False) and cut(N, 70, H, dk, dv, dtype, True)
    q, k, v, _, starts, at, state, g = mixer_inputs(lengths, H, dk, dv, dtype)
    decay = torch.tensor([-1e-3, -0.05, 0.0, -4e-4], device="cuda")
    do, dstate = randn(g, *v.shape, dtype=dtype), randn(g, *state.shape)
    terms = max(dk, dv) + 64 + 4 * (max(lengths) // 32 + 1)
    for st, ds in ((state, dstate), (None, None)):
        o, last = gr.linear_attention(q, k, v, decay, 0.3, seq_starts=starts, state=st)
        o64, l64 = ref.recurrence(q, k, v, decay, 0.3, at, st)
        om, lm = ref.recurrence(q, k, v, decay, 0.3, at, st, magnitudes=True)
        within(o, o64, mixer_bounds(o64, om, terms, dtype), "o")
        within(last, l64, (terms + 64) * U32 * lm, "state")
        got = gr.linear_attention_backward(do, q, k, v, decay, 0.3, seq_starts=starts, state=st, dstate=ds)
        want = ref.recurrence_grad(do, q, k, v, decay, 0.3, at, st, ds)
        mags = ref.recurrence_grad(do, q, k, v, decay, 0.3, at, st, ds, magnitudes=True)
        assert rel(o, o64) <= tol
        for name, a, b, m in zip(("dq", "dk", "dv"), got, want, mags):
            within(a, b, mixer_bounds(b, m, terms, dtype) + (2 ** -16 * m if dtype == BF else 0), name)
            assert rel(a, b) <= tol, name
        if ds is not None:
            within(got[3], want[3], (terms + 64) * U32 * mags[3], "dstate_in")


@pytest.mark.parametrize("lengths,H,with_state", [([70, 150, 9, 40], 2, True), ([70, 300, 9, 140], 6, True),
                                                  ([70, 300, 9, 140], 6, False), ([70, 2000, 9, 140], 2, True),
                                                  ([70, 2000, 9, 140], 2, False)])
@pytest.mark.parametrize("dk,dv,dtype", [(128, 128, BF), (64, 64, BF), (64, 128, BF), (64, 64, F32)])
def test_linear_attention_gradient_nothing_leaks(lengths, H, with_state, dk, dv, dtype):
    """What is not finite reaches only the gradients that it is a part of: through the past of dq, the future of dk and
    dv, never another sequence or head. In the middle of a sequence (of several chunks and segments), and in the rows
    right behind and before another one's end."""
    if H == 6:
        above_few_rows(lengths, H)
    if lengths[1] == 2000:
        assert cut(sum(lengths), 4, H, dk, dv, dtype, True)
    q, k, v, _, starts, at, state, g = mixer_inputs(lengths, H, dk, dv, dtype, layout="plain")
    decay = -torch.exp2(-torch.linspace(3.0, 12.0, H, device="cuda"))
    do, dstate = randn(g, *v.shape, dtype=dtype), randn(g, *state.shape)
    if not with_state:
        state = dstate = None
    clean = {"do": do, "q": q, "k": k, "v": v}

    def grads(a, **kw):
        return gr.linear_attention_backward(a["do"], a["q"], a["k"], a["v"], decay, 0.3, **kw)

    want = grads(clean, seq_starts=starts, state=state, dstate=dstate)
    for value in (float("nan"), float("inf")):
        for seq, t in ((1, at[1] + lengths[1] // 2), (1, at[1]), (1, at[2] - 1), (3, at[3] + 1)):
            past, future = (at[seq], t + 1), (t, at[seq + 1])      # rows whose future, past holds t
            own = (t, t + 1)
            hits = {"do": (own, past, past), "q": (None, past, past), "k": (future, None, own), "v": (future, own, None)}
            for name, hit in hits.items():
                args = dict(clean)
                args[name] = clean[name].clone()
                args[name][t, 1, 5] = value
                got = grads(args, seq_starts=starts, state=state, dstate=dstate)
                for what, a, b, rows in zip(("dq", "dk", "dv"), got, want, hit):
                    touched = torch.zeros(len(q), H, dtype=torch.bool, device="cuda")
                    if rows is not None:
                        touched[rows[0]:rows[1], 1] = True
                    assert torch.equal(a[~touched], b[~touched]), (name, what, t)
                    if rows is not None:
                        assert not torch.isfinite(a[t, 1]).all(), (name, what, t)
                if with_state:
                    keep = torch.ones(len(lengths), H, dtype=torch.bool, device="cuda")
                    keep[seq, 1] = name in ("k", "v")
                    assert torch.equal(got[3][keep], want[3][keep]), (name, t)
    # rows that no sequence holds are not read into one and not written
    args = {name: t.clone() for name, t in clean.items()}
    for t in args.values():
        t[at[3]:] = float("nan")
    out = [torch.full_like(t, 7.0) for t in want[:3]]
    part = None if state is None else state[:3].contiguous()
    dpart = None if dstate is None else dstate[:3].contiguous()
    grads(args, seq_starts=starts[:4].contiguous(), state=part, dstate=dpart, out=out)
    for a in out:
        assert (a[at[3]:] == 7).all() and torch.isfinite(a[:at[3]]).all()
