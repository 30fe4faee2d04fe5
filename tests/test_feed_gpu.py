"""GPU parity of the gated feed-forward sublayer, its gradient, FP8 blocks and their product against their
64-bit definitions, elementwise within the bounds of tests/feed_ref.py."""
from __future__ import annotations

import pytest
import torch

import feed_ref as ref
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


def randn(seed, *shape, std=1.0, dtype=F32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def within(got, want, bound, what):
    assert torch.isfinite(got.float()).all(), what
    over = ((got.double() - want).abs() - bound).max().item() if want.numel() else -1.0
    assert over <= 0, f"{what}: {over:.3e} over the bound"


def weights(D, F, dtype, seed=0):
    return randn(seed + 1, 2, F, D, std=D ** -0.5, dtype=dtype), randn(seed + 2, D, F, std=F ** -0.5, dtype=dtype)


# tokens, d_model, d_ff: single tokens, ends inside every tile, both sides of each rule on sizes
SIZES = [(1, 8, 8), (1, 256, 1024), (2, 2560, 1288), (5, 72, 4104), (16, 64, 128), (17, 136, 520), (33, 1000, 2728),
         (64, 512, 256), (127, 128, 640), (128, 264, 264), (129, 256, 2048), (200, 1032, 136), (256, 4096, 256),
         (257, 256, 512), (300, 2560, 1288), (511, 136, 3336), (700, 384, 1024), (1025, 512, 1160), (2305, 520, 776),
         (4099, 264, 1032), (3400, 1160, 1160), (301, 1800, 2056),
         # long sums: few tiles, and the tiles behind whole waves of them, divided along k
         (600, 7168, 256), (600, 256, 7168), (7000, 264, 520), (5000, 7168, 512)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_forward(i, dtype):
    N, D, F = SIZES[i]
    name = ("silu", "gelu")[i % 2]
    x, (w_in, w_out) = randn(i, N, D, std=1.5, dtype=dtype), weights(D, F, dtype, i)
    y = gr.feed_forward(x, w_in, w_out, name)
    y2, pre = gr.feed_forward(x, w_in, w_out, name, keep=True)
    wy, wp, by, bp = ref.forward(x, w_in, w_out, name, dtype)
    within(pre, wp, bp, "pre")
    within(y2, wy, by, "y")
    assert torch.equal(y, y2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_backward(i, dtype):
    N, D, F = SIZES[i]
    name = ("gelu", "silu")[i % 2]
    x, (w_in, w_out) = randn(i, N, D, std=1.5, dtype=dtype), weights(D, F, dtype, i)
    dy, pre = randn(50 + i, N, D, dtype=dtype), randn(90 + i, N, 2, F, std=1.5, dtype=dtype)
    got = gr.feed_forward_backward(dy, x, w_in, w_out, pre, name)
    for g, (want, bound), what in zip(got, ref.backward(dy, x, w_in, w_out, pre, name, dtype),
                                      ("dx", "dw_in", "dw_out")):
        within(g, want, bound, what)


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_gradient_matches_differences(name):
    """The gradients along random directions against central differences of the 64-bit forward pass. The step is
    2^-10: the difference's own error is its third derivative's, step^2 / 6 of terms of the gradient's size."""
    N, D, F = 37, 64, 136
    x, (w_in, w_out) = randn(1, N, D), weights(D, F, F32)
    dy = randn(3, N, D)
    _, pre = gr.feed_forward(x, w_in, w_out, name, keep=True)
    grads = gr.feed_forward_backward(dy, x, w_in, w_out, pre, name)

    def loss(*p):
        x, w_in, w_out = p
        h = ref.act(x @ w_in[0].T, name)[0] * (x @ w_in[1].T)
        return ((h @ w_out.T) * dy.double()).sum().item()

    at, step = [t.double() for t in (x, w_in, w_out)], 2.0 ** -10
    for k, g in enumerate(grads):
        way = randn(7 + k, *g.shape).double()
        ahead, behind = ([p + s * step * way if j == k else p for j, p in enumerate(at)] for s in (1, -1))
        want = (loss(*ahead) - loss(*behind)) / (2 * step)
        got = (g.double() * way).sum().item()
        assert abs(got - want) <= 1e-4 * (g.double().norm() * way.norm()).item(), k


def test_no_tokens():
    w_in, w_out = weights(64, 128, BF)
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    y, pre = gr.feed_forward(x, w_in, w_out, keep=True)
    assert y.shape == (0, 64) and pre.shape == (0, 2, 128)
    dx, dw_in, dw_out = gr.feed_forward_backward(x, x, w_in, w_out, pre, dw_in=torch.full_like(w_in, 7),
                                                 dw_out=torch.full_like(w_out, 7))
    assert dx.shape == x.shape and not dw_in.any() and not dw_out.any()
    eight = gr.fp8_encode_blocks(w_in, 128), gr.fp8_encode_blocks(w_out, 128)
    assert gr.feed_forward_fp8(x, *eight).shape == x.shape
    codes, scales = gr.fp8_encode_blocks(x)
    assert codes.shape == (0, 64) and scales.shape == (0, 1)
    assert gr.fp8_matmul((codes, scales), gr.fp8_encode_blocks(w_in[0], 128)).shape == (0, 128)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("N", [3, 400])
def test_what_is_not_finite_stays_in_its_rows(N, value):
    D, F = 256, 520
    x, (w_in, w_out) = randn(1, N, D, dtype=BF), weights(D, F, BF)
    clean = gr.feed_forward(x, w_in, w_out)
    x[1, 77] = value
    y = gr.feed_forward(x, w_in, w_out)
    assert not torch.isfinite(y[1]).any()
    keep = torch.arange(N, device="cuda") != 1
    assert torch.equal(y[keep], clean[keep])


# ---- FP8 ----------------------------------------------------------------------------------------

def wild(seed, *shape, dtype):
    """Values over many powers of two, with zeros, blocks of zeros, ties and the edges of the exponents."""
    m = randn(seed, *shape) * torch.exp2(12 * randn(seed + 1, *shape[:-1], 1))
    flat = m.view(-1, shape[-1])
    flat[0, :16] = 0
    if flat.shape[0] > 8:
        flat[1] = 0
        flat[2] *= 2.0 ** -100
        flat[3] = torch.arange(shape[-1], device="cuda") % 57 * 0.0625      # ties between codes
        flat[4, 0] = 448 * 2.0 ** 5
        flat[4, 1:] = 1.0
        flat[5] = 2.0 ** -130
        flat[6] = 3e38
        flat[7] = 449.0
    return m.to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("shape", [(1, 16), (1, 128), (3, 144), (128, 128), (129, 4096), (300, 1040), (1000, 272),
                                   (2, 136, 400), (3, 128, 256), (5, 1, 16)])
def test_encode_blocks(shape, rows, dtype):
    m = wild(len(shape) + shape[-1], *shape, dtype=dtype)
    codes, scales = gr.fp8_encode_blocks(m, rows)
    want, e = ref.encode(m, rows)
    assert scales.dtype == codes.dtype == torch.uint8
    assert torch.equal(scales.double() - 127, e)
    assert torch.equal(codes.view(torch.float8_e4m3fn).double(), want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_encode_of_what_is_not_finite(value, rows, dtype):
    m = randn(1, 200, 272, dtype=dtype)
    clean = gr.fp8_encode_blocks(m, rows)
    m[131, 130] = value
    codes, scales = gr.fp8_encode_blocks(m, rows)
    hit = torch.zeros(200, 272, dtype=torch.bool, device="cuda")
    hit[(131 if rows == 1 else 128):(132 if rows == 1 else 200), 128:256] = True
    assert (codes[hit] == 0x7f).all() and torch.equal(codes[~hit], clean[0][~hit])
    at = scales == 255
    assert at.sum() == 1 and at[131 // rows, 1] and torch.equal(scales[~at], clean[1][~at])


@pytest.mark.parametrize("N,K,O", [(1, 16, 8), (1, 4096, 512), (3, 144, 136), (16, 128, 128), (17, 1040, 264),
                                   (64, 512, 1024), (100, 272, 2056), (128, 4096, 256), (129, 528, 520), (255, 2560, 128),
                                   (256, 640, 1032), (257, 1168, 384), (600, 512, 2560), (1111, 1040, 1288),
                                   (3000, 656, 776), (3400, 400, 1160), (3400, 1040, 1096), (600, 16384, 264),
                                   (5000, 12288, 1032)])
def test_fp8_matmul(N, K, O):
    a = gr.fp8_encode_blocks(randn(N, N, K) * torch.exp2(3 * randn(K, N, 1)))
    b = gr.fp8_encode_blocks(randn(O, O, K) * torch.exp2(2 * randn(1, -(-O // 128), 1)).repeat_interleave(128, 0)[:O],
                             128)
    out = gr.fp8_matmul(a, b)
    want, bound = ref.product(a, b)
    within(out, want, bound, "out")


@pytest.mark.parametrize("N", [1, 40, 300, 512, 900])
def test_fp8_matmul_of_scales_at_any_address(N):
    """The same bits whether the scales' rows are read as they lie or laid out first."""
    K, O = 1024, 264
    a = gr.fp8_encode_blocks(randn(1, N, K) * torch.exp2(3 * randn(2, N, 1)))
    b = gr.fp8_encode_blocks(randn(3, O, K), 128)
    want = gr.fp8_matmul(a, b)

    def moved(t):
        return torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)

    for pa, pb in ((a, (b[0], moved(b[1]))), ((a[0], moved(a[1])), b)):
        assert torch.equal(gr.fp8_matmul(pa, pb), want)


def test_fp8_matmul_of_nan_blocks():
    """A NaN exponent reaches the outputs of its rows and no others, in either operand."""
    for N in (5, 300):
        x, w = randn(1, N, 400), randn(2, 384, 400)
        clean = gr.fp8_matmul(gr.fp8_encode_blocks(x), gr.fp8_encode_blocks(w, 128))
        x[3, 200] = float("inf")
        w[140, 399] = float("nan")
        out = gr.fp8_matmul(gr.fp8_encode_blocks(x), gr.fp8_encode_blocks(w, 128))
        bad = torch.zeros_like(out, dtype=torch.bool)
        bad[3], bad[:, 128:256] = True, True
        assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("i,size", list(enumerate([
    (1, 16, 16), (1, 256, 1024), (3, 2560, 1296), (16, 64, 128), (33, 144, 400), (64, 1024, 512), (127, 272, 640),
    (128, 512, 272), (200, 1040, 2064), (257, 256, 512), (500, 528, 784), (1030, 384, 1168), (2300, 272, 656), (4400, 1168, 1040), (600, 12288, 272),
    (600, 272, 12288)])))
def test_feed_forward_fp8(i, size):
    N, D, F = size
    name = ("silu", "gelu")[i % 2]
    x = randn(i, N, D, std=1.5, dtype=BF) * (1 + 30 * (torch.arange(D, device="cuda") % 61 == 7)).to(BF)
    w_in, w_out = weights(D, F, F32, i)
    w_in, w_out = gr.fp8_encode_blocks(w_in, 128), gr.fp8_encode_blocks(w_out, 128)
    y = gr.feed_forward_fp8(x, w_in, w_out, name)
    want, bound = ref.forward_fp8(x, w_in, w_out, name)
    within(y, want, bound, "y")


@pytest.mark.parametrize("N", [3, 700])
def test_feed_forward_fp8_keeps_what_is_not_finite_in_its_rows(N):
    D, F = 272, 656
    x, (w_in, w_out) = randn(1, N, D, dtype=BF), weights(D, F, F32)
    w_in, w_out = gr.fp8_encode_blocks(w_in, 128), gr.fp8_encode_blocks(w_out, 128)
    clean = gr.feed_forward_fp8(x, w_in, w_out)
    x[1, 77] = float("inf")
    y = gr.feed_forward_fp8(x, w_in, w_out)
    assert torch.isnan(y[1]).all()
    keep = torch.arange(N, device="cuda") != 1
    assert torch.equal(y[keep], clean[keep])


def test_rows_past_32_bits():
    """pre, h and their gradients pass 2^31 elements: the last rows against the definition, and the weights'
    gradients of rows that are zero but for those."""
    N, D, F = 70_001, 64, 16_384
    w_in, w_out = weights(D, F, BF)
    x = torch.zeros(N, D, dtype=BF, device="cuda")
    x[-300:] = randn(1, 300, D, dtype=BF)
    y, pre = gr.feed_forward(x, w_in, w_out, keep=True)
    wy, wp, by, bp = ref.forward(x[-300:], w_in, w_out, "silu", BF)
    within(y[-300:], wy, by, "y")
    within(pre[-300:], wp, bp, "pre")
    assert not y[:-300].any() and not pre[:-300].any()
    dx, dw_in, dw_out = gr.feed_forward_backward(x, x, w_in, w_out, pre)
    want = ref.backward(x[-300:], x[-300:], w_in, w_out, pre[-300:], "silu", BF)
    within(dx[-300:], *want[0], "dx")
    assert not dx[:-300].any()
    # the other rows add zeros, which leave every partial sum as it is
    within(dw_in, *want[1], "dw_in")
    within(dw_out, *want[2], "dw_out")
    eight = gr.fp8_encode_blocks(w_in, 128), gr.fp8_encode_blocks(w_out, 128)
    y = gr.feed_forward_fp8(x, *eight)
    wy, by = ref.forward_fp8(x[-300:], *eight, "silu")
    within(y[-300:], wy, by, "y")
    assert not y[:-300].any()


# ---- how calls are made -------------------------------------------------------------------------

def every_call(N, D=256, F=640):
    """[(name, () -> outputs)] on one set of inputs."""
    x, dy, (w_in, w_out) = randn(1, N, D, dtype=BF), randn(2, N, D, dtype=BF), weights(D, F, BF)
    pre = randn(3, N, 2, F, dtype=BF)
    e_in, e_out, a = gr.fp8_encode_blocks(w_in, 128), gr.fp8_encode_blocks(w_out, 128), gr.fp8_encode_blocks(dy)
    b = gr.fp8_encode_blocks(w_in.flatten(0, 1), 128)
    return [("feed_forward", lambda **kw: gr.feed_forward(x, w_in, w_out, keep=True, **kw)),
            ("feed_forward_backward", lambda **kw: gr.feed_forward_backward(dy, x, w_in, w_out, pre, **kw)),
            ("fp8_encode_blocks", lambda **kw: gr.fp8_encode_blocks(x, **kw)),
            ("fp8_matmul", lambda **kw: (gr.fp8_matmul(a, b, **kw),)),
            ("feed_forward_fp8", lambda **kw: (gr.feed_forward_fp8(x, e_in, e_out, **kw),))]


@pytest.mark.parametrize("N", [7, 300, 1500])
@pytest.mark.parametrize("i", range(5))
def test_repeats_streams_and_graphs(i, N):
    """The same bits again, on another stream, and from a graph that is replayed beside eager calls."""
    name, call = every_call(N)[i]
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        own = call()
    given = call(stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = call()
    for t in captured:
        t.zero_()
    graph.replay()
    again = call()
    graph.replay()
    torch.cuda.synchronize()
    for other in (own, given, captured, again):
        assert all(torch.equal(a, b) for a, b in zip(want, other)), name


@pytest.mark.parametrize("N", [1, 64, 300])
def test_nothing_is_written_behind_the_outputs(N):
    """Outputs inside larger buffers: what lies before and behind them stays."""
    D, F, pad = 136, 264, 512
    x, dy, (w_in, w_out) = randn(1, N, D, dtype=BF), randn(2, N, D, dtype=BF), weights(D, F, BF)
    pre = randn(3, N, 2, F, dtype=BF)

    def framed(*shape):
        n = 1
        for s in shape:
            n *= s
        buf = torch.full((n + 2 * pad,), 5.0, dtype=BF, device="cuda")
        return buf, buf[pad:pad + n].view(shape)

    made = [framed(N, D), framed(N, 2, F), framed(N, D), framed(2, F, D), framed(D, F)]
    y, p, dx, dwi, dwo = (t for _, t in made)
    feed = gr._FEED.pack(N, D, F, gr.GR_BF16, 0)
    for gradient in (0, 1):
        need = gr._need("gr_feed_workspace_size", feed, gradient)
        ws = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
        if gradient:
            gr.feed_forward_backward(dy, x, w_in, w_out, pre, dx=dx, dw_in=dwi, dw_out=dwo, workspace=ws[:need])
        else:
            gr.feed_forward(x, w_in, w_out, y=y, pre=p, workspace=ws[:need])
        assert (ws[need:] == 77).all()
    for buf, t in made:
        assert (buf[:pad] == 5).all() and (buf[pad + t.numel():] == 5).all()


def test_a_workspace_that_is_too_small_is_refused():
    x, (w_in, w_out) = randn(1, 300, 256, dtype=BF), weights(256, 640, BF)
    with pytest.raises(gr.GRError):
        gr.feed_forward(x, w_in, w_out, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


def test_wrong_arguments_are_refused():
    x, (w_in, w_out) = randn(1, 4, 64, dtype=BF), weights(64, 128, BF)
    ok = dict(x=x, w_in=w_in, w_out=w_out)
    for bad in (dict(x=x.float()), dict(x=x[:, :32]), dict(w_in=w_in[0]), dict(w_in=w_in.transpose(1, 2)),
                dict(w_out=w_out.T), dict(activation="relu"), dict(y=x[:2]), dict(w_out=w_out.cpu())):
        with pytest.raises(ValueError):
            gr.feed_forward(**{**ok, **bad})
    with pytest.raises(gr.GRError):
        gr.feed_forward(x, w_in, w_out, y=x)
    e, o = gr.fp8_encode_blocks(w_in, 128), gr.fp8_encode_blocks(w_out, 128)
    for bad in ((x.float(), e, o), (x, o, o), (x, (e[0], e[1][:1]), o), (x, e, (o[0], o[1].int()))):
        with pytest.raises(ValueError):
            gr.feed_forward_fp8(*bad)
    for bad in ((w_in, 64), (w_in.half(), 1), (w_in[0, 0], 1)):
        with pytest.raises(ValueError):
            gr.fp8_encode_blocks(*bad)
    with pytest.raises(gr.GRError):
        gr.fp8_encode_blocks(torch.zeros(4, 24, device="cuda"))


@pytest.mark.parametrize("N", [5, 900])
@pytest.mark.parametrize("i", range(5))
def test_two_streams_at_once(i, N):
    """Calls under way on two streams at the same time, each with memory of its own."""
    name, call = every_call(N, 512, 1280)[i]
    want = call()
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(12):
        for side in sides:
            with torch.cuda.stream(side):
                got.append(call())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for outs in got for a, b in zip(outs, want)), name


@pytest.mark.parametrize("N", [1, 60, 700])
def test_weights_written_just_before_a_call(N):
    """Weights are read ahead of the products' own predecessors, but not of what wrote them."""
    D, F = 1024, 4096
    x = randn(1, N, D, dtype=BF)
    sets = [weights(D, F, BF, seed) for seed in (3, 9)]
    eights = [tuple(gr.fp8_encode_blocks(w, 128) for w in s) for s in sets]
    want = [gr.feed_forward(x, *s) for s in sets]
    want8 = [gr.feed_forward_fp8(x, *e) for e in eights]
    w = [t.clone() for t in sets[0]]
    e = [tuple(t.clone() for t in pair) for pair in eights[0]]
    got, got8 = [], []
    for k in range(10):
        for to, new in zip(w, sets[k % 2]):
            to.copy_(new)
        got.append(gr.feed_forward(x, *w))
        for pair, new in zip(e, eights[k % 2]):
            for to, t in zip(pair, new):
                to.copy_(t)
        got8.append(gr.feed_forward_fp8(x, *e))
    for k in range(10):
        assert torch.equal(got[k], want[k % 2]) and torch.equal(got8[k], want8[k % 2]), k


def test_results_do_not_depend_on_what_the_workspace_holds():
    """Workspaces and outputs full of NaN bytes before the call, for every way a call can be divided."""
    for N in (3, 300, 700, 2305):
        for name, call in every_call(N, 1032 - 8, 2064):
            want = call()
            torch.cuda.synchronize()
            kept = torch.empty
            try:
                torch.empty = lambda *a, **k: kept(*a, **k).view(torch.uint8).fill_(255).view(k["dtype"]) \
                    if k.get("dtype") != torch.uint8 else kept(*a, **k).fill_(255)
                again = call()
            finally:
                torch.empty = kept
            assert all(torch.equal(a, b) for a, b in zip(want, again)), (name, N)
