"""Where the feed-forward sublayer's arithmetic is most easily lost: the normal distribution far below zero, and sums
over very many tokens. Inputs are chosen so that everything else is exact, and every bound is relative to the value."""
from __future__ import annotations

import math

import pytest
import torch

from stream_gated_residual_gb300 import gr

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
ULP = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    gr.load()
    gr.device_status(clear=True)
    yield
    torch.cuda.empty_cache()
    assert gr.device_status() == 0


# ---- GELU far below zero --------------------------------------------------------------------------
#
# fp32: Φ(g) = erfc(x) / 2 at x = -g / sqrt 2. x is off by two roundings, 2^-23 of itself, and erfc(x) by |x erfc'(x) /
# erfc(x)| <= 2 x^2 + 1 = g^2 + 1 times that, beside erfcf's own 4 units; two products follow: (g^2 + 8)·2^-23 of g Φ(g)
# covers them and the multiplication by up. bf16 and FP8: exp(-g^2 / 2) times a polynomial in t = 1 / (1 + 0.28 |g|) that is
# within 1.7e-7: the exponent's rounding g^2 / 4 units, the hardware's exponential 2 + 0.59 g^2, the polynomial, t and the
# products 8 more, of which the last three are those above: (g^2 + 8)·2^-23 again. The slope is Φ + g φ, φ's exponential off
# by as much as that (fp32: g^2 / 4 + 2 units); the two terms are at least 8 : 1 apart for g <= -3, so (2 g^2 + 16)·2^-23
# covers it everywhere.

def tail(N, dtype):
    """Gates in [-10, -3], ends included, as the dtype holds them."""
    return -torch.linspace(3, 10, N, device="cuda").to(dtype)


def relative(got, want, bound, what):
    over = ((got.double() - want).abs() / want.abs() - bound).max().item()
    assert over <= 0, f"{what}: {over:.3e} over the bound, relative"


def gelu(g):
    """(g Φ(g), its slope) in 64 bits."""
    g = g.double()
    below = 0.5 * torch.special.erfc(-g / math.sqrt(2))
    return g * below, below + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


@pytest.mark.parametrize("N", [3, 200, 701])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_gelu_far_below_zero(dtype, N):
    """x = (g, 1), W_g takes the first, W_u the second, W_o is the identity: y[n][d] = g Φ(g) of row n. h and y are
    rounded to the dtype once each."""
    D, g = 64, tail(N, dtype)
    x = torch.zeros(N, D, dtype=dtype, device="cuda")
    x[:, 0], x[:, 1] = g, 1
    w_in = torch.zeros(2, D, D, dtype=dtype, device="cuda")
    w_in[0, :, 0], w_in[1, :, 1] = 1, 1
    y, pre = gr.feed_forward(x, w_in, torch.eye(D, dtype=dtype, device="cuda"), "gelu", keep=True)
    assert torch.equal(pre[:, 0], g[:, None].expand(N, D))
    assert (pre[:, 1] == 1).all()
    bound = (g.double() ** 2 + 8) * ULP + (2 * 2.0 ** -8 + 2.0 ** -15 if dtype == BF else 0)
    relative(y, gelu(g)[0][:, None].expand(N, D), bound[:, None], "y")


@pytest.mark.parametrize("N", [3, 200, 701])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_gelu_gradient_far_below_zero(dtype, N):
    """dh is 1 in the first channel and 0 in the others, up is 1: dx = (f'(g), g Φ(g)), dW_o's first row Σ h."""
    D, g = 64, tail(N, dtype)
    dy, w_out = (torch.zeros(n, D, dtype=dtype, device="cuda") for n in (N, D))
    dy[:, 0], w_out[0, 0] = 1, 1
    w_in = torch.zeros(2, D, D, dtype=dtype, device="cuda")
    w_in[0, 0, 0], w_in[1, 0, 1] = 1, 1
    pre = torch.ones(N, 2, D, dtype=dtype, device="cuda")
    pre[:, 0] = g[:, None]
    x = torch.ones(N, D, dtype=dtype, device="cuda")
    dx, dw_in, dw_out = gr.feed_forward_backward(dy, x, w_in, w_out, pre, "gelu")
    a, slope = gelu(g)
    bound = (2 * g.double() ** 2 + 16) * ULP + (2 * 2.0 ** -8 + 2.0 ** -15 if dtype == BF else 0)
    relative(dx[:, 0], slope, bound, "dx, gate")
    relative(dx[:, 1], a, bound, "dx, up")
    # sums of terms of one sign, each off by its own bound; the sum itself by (N + 4) units
    worst = bound.max().item() + (N + 4) * ULP
    relative(dw_out[0], a.sum().expand(D), worst, "dw_out")
    relative(dw_in[1, 0], a.sum().expand(D), worst, "dw_in, up")
    relative(dw_in[0, 0], slope.sum().expand(D), worst, "dw_in, gate")


@pytest.mark.parametrize("N", [15, 600])
def test_gelu_far_below_zero_in_fp8(N):
    """The gates lie on the e4m3 grid and the weights are 0 and 1, so both are encoded as they are. h is the same in
    all 128 channels of a token and rounded to a code, by at most 2^-4 of it, which y holds exactly."""
    D = 128
    g = -torch.tensor([3, 3.25, 3.5, 3.75, 4, 4.5, 5, 5.5, 6, 6.5, 7, 7.5, 8, 9, 10], device="cuda").repeat(N // 15)
    x = torch.zeros(N, D, dtype=BF, device="cuda")
    x[:, 0], x[:, 1] = g, 1
    w_in = torch.zeros(2, D, D, device="cuda")
    w_in[0, :, 0], w_in[1, :, 1] = 1, 1
    y = gr.feed_forward_fp8(x, gr.fp8_encode_blocks(w_in, 128), gr.fp8_encode_blocks(torch.eye(D, device="cuda"), 128),
                            "gelu")
    bound = (g.double() ** 2 + 8) * ULP
    relative(y, gelu(g)[0][:, None].expand(N, D), (2.0 ** -4 * (1 + bound) + bound)[:, None], "y")


# ---- fp32 operands of any size --------------------------------------------------------------------

@pytest.mark.parametrize("power", [0, -60, -100, -110, -120, -126, 60, 90])
def test_fp32_products_of_small_and_large_operands(power):
    """An operand is held as three bf16 terms: to 2^-24 of it, but to no less than 2^-134, half of bf16's last place. dy
    of size 2^power against h of size 1: dW_o = dyᵀ h within the bound of sums of N products, (N + 4) units of the sum of
    magnitudes, which covers h's own error beside it (16 units), and 2^-134 Σ |h|."""
    N, D, F = 300, 64, 136
    gen = torch.Generator(device="cuda")
    gen.manual_seed(power + 200)
    dy, x, w_in, w_out, pre = (torch.randn(*shape, generator=gen, device="cuda")
                               for shape in ((N, D), (N, D), (2, F, D), (D, F), (N, 2, F)))
    dy *= 2.0 ** power
    dw_out = gr.feed_forward_backward(dy, x, w_in, w_out, pre)[2]
    gate, up = pre.double().unbind(1)
    h = gate * torch.sigmoid(gate) * up
    size = dy.double().abs().T @ h.abs()
    bound = (N + 20) * ULP * size + 2.0 ** -134 * h.abs().sum(0)
    assert ((dw_out.double() - dy.double().T @ h).abs() <= bound).all()


# ---- sums over very many tokens -------------------------------------------------------------------

def test_one_signed_sums_over_a_million_tokens():
    """The weights' gradients of 2^20 tokens, all terms of one sign. h = 16 u (GELU of 16 is 16, u a power of two),
    dh = dy's first channel, dgate = dh u and dup = 16 dh are exact in bf16, so
        dW_o[d][f] = 16 u_f Σ dy[n][d],   dW_u[f][d] = 16 Σ dy[n][0] x[n][d],   dW_g[f][d] = u_f Σ dy[n][0] x[n][d].
    The result's rounding is off by 2^-8. An accumulator takes up to 1024 blocks of 64 k, 2^12 additions of 16 products each,
    which are cut to its last place with three guard bits at least: up to two units, 2^-22, of the sum so far, which is
    half of the last one on average: 2^-11. The parts' sums add a few units. The 2304 sums of each kind are spread evenly
    over an octave, so their roundings, of deviation 2^-8 / sqrt(3), average to zero within four times 2^-8 /
    sqrt(3 · 2304) < 2^-12. (One accumulator for all of k would add 2^16 cuts.)"""
    N, D, F = 1 << 20, 2304, 1792

    def some(seed):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        v = torch.rand(N, D, generator=gen, device="cuda", dtype=F32).add_(0.5)
        return v.mul_(torch.linspace(1, 2, D, device="cuda")).to(BF)

    x, dy = some(1), some(2)
    u = torch.exp2((torch.arange(F, device="cuda") % 4 - 1).float())
    pre = torch.empty(N, 2, F, dtype=BF, device="cuda")
    pre[:, 0], pre[:, 1] = 16, u.to(BF)
    w_in = torch.zeros(2, F, D, dtype=BF, device="cuda")
    w_out = torch.zeros(D, F, dtype=BF, device="cuda")
    w_out[0] = 1
    dx, dw_in, dw_out = gr.feed_forward_backward(dy, x, w_in, w_out, pre, "gelu")
    assert not dx.any()
    del dx, pre
    each = [torch.stack([(x[at:at + 65536].double() * dy[at:at + 65536, :1].double()).sum(0),
                         dy[at:at + 65536].double().sum(0)]) for at in range(0, N, 65536)]
    xy, total = torch.stack(each).sum(0)
    for got, want, what in ((dw_out, 16 * total[:, None] * u.double(), "dw_out"),
                            (dw_in[0], u.double()[:, None] * xy, "dw_in, gate"),
                            (dw_in[1], (16 * xy)[None].expand(F, D), "dw_in, up")):
        off = (got.double() - want) / want
        print(f"{what}: {off.mean().item():.3e} on average, {off.abs().max().item():.3e} at most")
        assert off.abs().max().item() <= 2.0 ** -8 + 2.0 ** -11, what
        assert off.mean().abs().item() <= 2.0 ** -11 + 2.0 ** -12, what
