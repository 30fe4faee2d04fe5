"""The feed-forward products in the ways a call can be divided: whole tiles with a tail in parts behind them, in every
kind of product, the fp32 form, chunks of k; results against 64 bits, the same bits again in other circumstances, and
nothing written outside the outputs. That a size is divided as meant is read from its workspace: only parts take more than
the operands."""
from __future__ import annotations

import pytest
import torch

import feed_ref as ref
from stream_gated_residual_gb300 import gr
from test_feed_gpu import randn, weights, within

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    gr.load()
    gr.device_status(clear=True)
    yield
    torch.cuda.empty_cache()
    assert gr.device_status() == 0


# ---- how calls are divided ------------------------------------------------------------------------

def up(n, to):
    return -(-n // to) * to


def scales(rows, k):
    """Bytes of a product's scales of `rows` tokens, and of the weights' [rows][k]: words of four blocks."""
    words = -(-k // 512)
    return up(rows, 128) // 128 * words * 512, up(rows, 128) // 128 * words * 4


def parts(op, N, D, F):
    """Bytes of the parts in a call's workspace (fp8_matmul: D is K and F is O)."""
    if op == "fp8_matmul":
        need = gr._need("gr_fp8_matmul_workspace_size", gr._PRODUCT.pack(N, D, F))
        rest = (scales(N, D)[0], scales(F, D)[1])
    else:
        dtype = gr.GR_FP8 if op == "feed_forward_fp8" else gr.GR_BF16
        need = gr._need("gr_feed_workspace_size", gr._FEED.pack(N, D, F, dtype, 0), int(op == "feed_forward_backward"))
        if op == "feed_forward_fp8":
            rest = (N * D, scales(N, D)[0], N * F, scales(N, F)[0], 2 * scales(F, D)[1], scales(D, F)[1])
        else:
            rest = (2 * N * F,) + ((4 * N * F,) if op == "feed_forward_backward" else ())
    return need - sum(up(n, 256) for n in rest)


# (call, N, D, F, tiles and blocks of k of the one product that has a tail in parts behind whole tiles)
TAILS = {
    "h and pre": ("feed_forward", 5000, 7168, 512, 20 * 4, 112),
    "y": ("feed_forward", 2500, 2048, 7168, 10 * 8, 112),
    "dh": ("feed_forward_backward", 2800, 7168, 2048, 11 * 8, 112),
    "dw_in": ("feed_forward_backward", 8000, 1280, 2048, 16 * 5, 125),
    "fp8 product": ("fp8_matmul", 2500, 12288, 2048, 10 * 8, 96),
    "fp8 h": ("feed_forward_fp8", 600, 12288, 3456, 3 * 27, 96),
    "fp8 y": ("feed_forward_fp8", 2500, 2048, 12288, 10 * 8, 96),
}


def inputs(op, N, D, F, dtype=BF):
    """The call on inputs of its own: (() -> outputs, its tensors)."""
    if op == "fp8_matmul":
        a = gr.fp8_encode_blocks(randn(1, N, D) * torch.exp2(3 * randn(2, N, 1)))
        b = gr.fp8_encode_blocks(randn(3, F, D), 128)
        return (lambda **kw: (gr.fp8_matmul(a, b, **kw),)), (a, b)
    x, (w_in, w_out) = randn(4, N, D, std=1.5, dtype=dtype), weights(D, F, dtype, 5)
    if op == "feed_forward_fp8":
        w_in, w_out = gr.fp8_encode_blocks(w_in, 128), gr.fp8_encode_blocks(w_out, 128)
        return (lambda **kw: (gr.feed_forward_fp8(x, w_in, w_out, **kw),)), (x, w_in, w_out)
    if op == "feed_forward":
        return (lambda **kw: gr.feed_forward(x, w_in, w_out, keep=True, **kw)), (x, w_in, w_out)
    dy, pre = randn(8, N, D, dtype=dtype), randn(9, N, 2, F, std=1.5, dtype=dtype)
    return (lambda **kw: gr.feed_forward_backward(dy, x, w_in, w_out, pre, **kw)), (dy, x, w_in, w_out, pre)


def close(got, want, terms, what):
    """The norm of the error: a lost or doubled product of a long sum shows here, where the elementwise bounds, which grow
    with k, would let it pass. `terms` is the norm of the operand's roundings, each at most 2^-8 and independent of the
    others, on their way to the result; the result's own is at most 2^-8 of it; 2^-11 is left for the sums."""
    off, size = (got.double() - want).norm().item(), want.norm().item()
    assert off <= 2.0 ** -8 * (size + terms) + 2.0 ** -11 * size, f"{what}: {off / size:.3e} of its norm"


@pytest.mark.parametrize("case", TAILS)
def test_a_tail_in_parts_behind_whole_tiles(case):
    op, N, D, F, tiles, blocks = TAILS[case]
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    if pairs == 76:
        assert 0 < tiles % pairs < pairs < tiles and blocks > 80
        # two partial tiles a pair: the tail of one product and of no other
        assert parts(op, N, D, F) == pairs * 2 * 256 * 256 * 4
    call, t = inputs(op, N, D, F)
    got = call()
    if op == "fp8_matmul":
        want, bound = ref.product(*t)
        within(got[0], want, bound, case)
        close(got[0], want, 0.0, case)
    elif op == "feed_forward_fp8":
        within(got[0], *ref.forward_fp8(*t, "silu"), case)
    elif op == "feed_forward":
        x, w_in, w_out = t
        wy, wp, by, bp = ref.forward(x, w_in, w_out, "silu", BF)
        within(got[0], wy, by, "y")
        within(got[1], wp, bp, "pre")
        h = ref.act(wp[:, 0], "silu")[0] * wp[:, 1]
        close(got[0], wy, (h.square() @ w_out.double().square().T).sum().sqrt().item(), "y")
        close(got[1], wp, 0.0, "pre")
    else:
        gradients_close(got, *t)


def gradients_close(got, dy, x, w_in, w_out, pre):
    dh = dy.double() @ w_out.double()
    a, slope = ref.act(pre[:, 0].double(), "silu")
    dpre = torch.cat([dh * pre[:, 1].double() * slope, dh * a], 1)
    h, flat = a * pre[:, 1].double(), w_in.double().flatten(0, 1)
    terms = [(dpre.square() @ flat.square()).sum(), (dpre.square().T @ x.double().square()).sum(),
             (dy.double().square().T @ h.square()).sum()]
    del dh, a, slope, dpre, h
    for g, (want, bound), e, what in zip(got, ref.backward(dy, x, w_in, w_out, pre, "silu", BF), terms,
                                         ("dx", "dw_in", "dw_out")):
        want, bound = (torch.stack(v) if isinstance(v, tuple) else v for v in (want, bound))
        within(g, want, bound, what)
        close(g, want, e.sqrt().item(), what)


def test_sums_over_tokens_in_chunks():
    """66000 tokens are 1032 blocks of 64, more than one accumulator takes: the 80 tiles of dW_in go in chunks of k, the 40
    of dW_out in even ranges, which are shorter."""
    op, N, D, F = "feed_forward_backward", 66_000, 1024, 2440
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        made = parts(op, N, D, F) // (256 * 256 * 4)
        assert made % 80 == 0 and 2 <= made // 80 <= 4
    call, t = inputs(op, N, D, F)
    gradients_close(call(), *t)


def test_sums_over_hidden_channels_in_chunks():
    """65544 hidden channels are 1025 blocks of 64 of the down product, 2049 of dx: y of 520 tokens in chunks of whole
    tiles, dx of 40 tokens, which are the product's columns, in chunks of theirs."""
    F = 65_544
    call, (x, w_in, w_out) = inputs("feed_forward", 520, 8192, F)
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        made = parts("feed_forward", 520, 8192, F) // (256 * 256 * 4)
        assert made % 96 == 0 and 2 <= made // 96 <= 4
    got, wp = call()[0], ref.forward(x, w_in, w_out, "silu", BF)
    h = ref.act(wp[1][:, 0], "silu")[0] * wp[1][:, 1]
    within(got, wp[0], wp[2], "y")
    close(got, wp[0], (h.square() @ w_out.double().square().T).sum().sqrt().item(), "y")
    del call, x, w_in, w_out, wp, h, got
    call, t = inputs("feed_forward_backward", 40, 12288, F)
    gradients_close(call(), *t)


@pytest.mark.parametrize("N,K,O", [(64, 7168, 2048), (600, 16384, 264), (8191, 7168, 520)])
def test_long_fp8_sums_lose_nothing(N, K, O):
    call, t = inputs("fp8_matmul", N, K, O)
    close(call()[0], ref.product(*t)[0], 0.0, "out")


@pytest.mark.parametrize("N,D,F", [(33, 7168, 264), (301, 1800, 2056), (700, 264, 4104)])
def test_long_fp32_sums_lose_nothing(N, D, F):
    """Three terms hold 2^-24 of an operand, the six products leave out 2^-24 of one each: some 2^-22 a product, which
    independent signs do not add up; 2^-20 of the norm is left for the sums' roundings."""
    call, (x, w_in, w_out) = inputs("feed_forward", N, D, F, F32)
    wy, wp, *_ = ref.forward(x, w_in, w_out, "silu", F32)
    for got, want in zip(call(), (wy, wp)):
        assert (got.double() - want).norm() <= 2.0 ** -19 * want.norm()


# ---- the same bits in every way of calling --------------------------------------------------------

WAYS = [(*TAILS[case][:4], BF) for case in ("h and pre", "dh", "fp8 h")] + \
       [("feed_forward", 7, 136, 264, F32), ("feed_forward", 700, 256, 640, F32), ("feed_forward_backward", 7, 136, 264, F32),
        ("feed_forward_backward", 700, 256, 640, F32), ("feed_forward_backward", 66_000, 1024, 2440, BF)]


@pytest.mark.parametrize("op,N,D,F,dtype", WAYS)
def test_repeats_streams_graphs_and_dirty_memory(op, N, D, F, dtype):
    """Again, on another stream, from a graph replayed beside eager calls, on two streams at once, and with workspaces
    and outputs full of NaN bytes."""
    call, _ = inputs(op, N, D, F, dtype)
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
    both = []
    for k in range(6):
        with torch.cuda.stream(side):
            both.append(call())
        both.append(call())
    torch.cuda.synchronize()
    kept = torch.empty
    try:
        torch.empty = lambda *a, **k: kept(*a, **k).view(torch.uint8).fill_(255).view(k["dtype"])
        dirty = call()
    finally:
        torch.empty = kept
    torch.cuda.synchronize()
    for other in (own, given, captured, again, dirty, *both):
        assert all(torch.equal(a, b) for a, b in zip(want, other))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("N", [3, 400])
def test_fp32_what_is_not_finite_stays_in_its_rows(N, value):
    D, F = 256, 520
    x, (w_in, w_out) = randn(1, N, D), weights(D, F, F32)
    dy, pre = randn(2, N, D), randn(3, N, 2, F)
    clean, dx = gr.feed_forward(x, w_in, w_out), gr.feed_forward_backward(dy, x, w_in, w_out, pre)[0]
    keep = torch.arange(N, device="cuda") != 1
    x[1, 77] = value
    y = gr.feed_forward(x, w_in, w_out)
    assert not torch.isfinite(y[1]).any() and torch.equal(y[keep], clean[keep])
    dy[1, 99] = value
    got = gr.feed_forward_backward(dy, x, w_in, w_out, pre)
    assert not torch.isfinite(got[0][1]).any() and torch.equal(got[0][keep], dx[keep])
    # a token that is not finite reaches the weights' gradients of its channels: x's 77th and dy's 99th
    assert not torch.isfinite(got[1][..., 77]).any() and not torch.isfinite(got[2][99]).any()


# ---- nothing outside the outputs ------------------------------------------------------------------

PAD = 512


def framed(dtype, *shape):
    """An output inside a larger buffer of one value."""
    n = 1
    for s in shape:
        n *= s
    buf = torch.full((n + 2 * PAD,), 5, dtype=dtype, device="cuda")
    return buf, buf[PAD:PAD + n].view(shape)


def frames_hold(made):
    for buf, t in made:
        assert (buf[:PAD] == 5).all() and (buf[PAD + t.numel():] == 5).all()


@pytest.mark.parametrize("op,N,D,F,dtype", [
    ("feed_forward", 700, 136, 264, BF), ("feed_forward", 1025, 520, 1160, BF), ("feed_forward", 300, 136, 264, F32),
    ("feed_forward_backward", 700, 136, 264, BF), ("feed_forward_backward", 1025, 520, 1160, BF),
    ("feed_forward_backward", 300, 136, 264, F32), ("feed_forward_backward", 66_000, 1032, 2440, BF),
    ("fp8_matmul", 3, 144, 136, BF), ("fp8_matmul", 700, 144, 136, BF), ("feed_forward_fp8", 5, 144, 272, BF),
    ("feed_forward_fp8", 700, 144, 272, BF), *((*TAILS[c][:4], BF) for c in TAILS)])
def test_nothing_is_written_outside_outputs_and_workspace(op, N, D, F, dtype):
    shapes = {"feed_forward": dict(y=(N, D), pre=(N, 2, F)),
              "feed_forward_backward": dict(dx=(N, D), dw_in=(2, F, D), dw_out=(D, F)),
              "fp8_matmul": dict(out=(N, F)), "feed_forward_fp8": dict(y=(N, D))}[op]
    made = {k: framed(dtype, *s) for k, s in shapes.items()}
    if op == "fp8_matmul":
        need = gr._need("gr_fp8_matmul_workspace_size", gr._PRODUCT.pack(N, D, F))
    else:
        code = gr.GR_FP8 if op == "feed_forward_fp8" else gr.GR_F32 if dtype == F32 else gr.GR_BF16
        need = gr._need("gr_feed_workspace_size", gr._FEED.pack(N, D, F, code, 0), int(op == "feed_forward_backward"))
    call, _ = inputs(op, N, D, F, dtype)
    ws = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    got = call(workspace=ws[:need], **{k: t for k, (_, t) in made.items()})
    assert (ws[need:] == 77).all()
    frames_hold(made.values())
    assert all(torch.equal(a, b) for a, b in zip(got, call()))


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("shape", [(5, 16), (129, 272), (2, 136, 400)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_encoder_writes_its_outputs_alone(shape, rows, dtype):
    m = randn(1, *shape, dtype=dtype)
    want = gr.fp8_encode_blocks(m, rows)
    made = [framed(torch.uint8, *t.shape) for t in want]
    got = gr.fp8_encode_blocks(m, rows, codes=made[0][1], scales=made[1][1])
    frames_hold(made)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---- more than 2^31 elements ----------------------------------------------------------------------

@pytest.mark.parametrize("op", ["feed_forward", "feed_forward_fp8"])
def test_hidden_values_past_32_bits(op):
    """h, and in FP8 its codes, pass 2^31 elements: the last rows against the definition; the rows before are zeros."""
    N, D, F = 140_032, 64, 16_384
    assert N * F > 1 << 31
    w_in, w_out = weights(D, F, BF)
    x = torch.zeros(N, D, dtype=BF, device="cuda")
    x[-768:] = randn(1, 768, D, dtype=BF)
    if op == "feed_forward":
        y = gr.feed_forward(x, w_in, w_out)
        want, _, bound, _ = ref.forward(x[-768:], w_in, w_out, "silu", BF)
    else:
        eight = gr.fp8_encode_blocks(w_in, 128), gr.fp8_encode_blocks(w_out, 128)
        y = gr.feed_forward_fp8(x, *eight)
        want, bound = ref.forward_fp8(x[-768:], *eight, "silu")
    within(y[-768:], want, bound, "y")
    assert not y[:-768].any()
