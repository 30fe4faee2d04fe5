"""The decoder with feed-forward sublayers: its gradients against torch autograd of the same model in 64 bits, its
token-by-token form against its prompt form, on bf16 and on FP8 weights, and the command that runs it."""
from __future__ import annotations

import math

import pytest
import torch

from stream_gated_residual_gb300 import decoder, gr
from stream_gated_residual_gb300.decoder import Config, Decoder

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    gr.load()


def plain_loss(cfg, p, log_decay, ids, targets, starts):
    """The model's loss from the formulas, on 64-bit CPU tensors that autograd follows."""
    H, d, N = cfg.heads, cfg.d_head, len(ids)
    seq = torch.searchsorted(starts, torch.arange(N), right=True)
    t = torch.arange(N)
    gap = t[:, None] - t[None, :]
    live = (gap >= 0) & (seq[:, None] == seq[None, :])
    decay = torch.where(live, torch.exp(log_decay[:, None, None] * gap.clamp(min=0)), 0.0)
    act = torch.nn.functional.silu if cfg.activation == "silu" else torch.nn.functional.gelu
    R = (math.sqrt(cfg.d_model) * p["embedding"][ids])[:, None].expand(-1, 4, -1)

    def read(R, at):
        n = R * p[f"{at}.gamma"] / (R.square().mean(-1, keepdim=True) + cfg.eps).sqrt()
        v = n.flatten(1)
        hidden = torch.nn.functional.silu(v @ p[f"{at}.w_down"].T / 4)
        G = torch.sigmoid(hidden @ p[f"{at}.w_up"].T).view_as(n)
        return (G * n).mean(1), 2 * torch.sigmoid(v @ p[f"{at}.w_write"].T / 4)

    for i in range(cfg.layers):
        x, s = read(R, f"{i}")
        q, k, u = (x @ p[f"{i}.qkv"].T).view(N, 3, H, d).unbind(1)
        scores = torch.einsum("nhd,mhd->hnm", q, k) * decay * d ** -0.5
        o = torch.einsum("hnm,mhd->nhd", scores, u)
        R = R + s[:, :, None] * (o.flatten(1) @ p[f"{i}.out"].T)[:, None]
        x, s = read(R, f"{i}.ff")
        gate, up = torch.einsum("nd,pfd->npf", x, p[f"{i}.ff.w_in"]).unbind(1)
        R = R + s[:, :, None] * ((act(gate) * up) @ p[f"{i}.ff.w_out"].T)[:, None]
    c = R - R.mean(-1, keepdim=True)
    z = c / (c.square().mean(-1, keepdim=True) + cfg.eps).sqrt() * p["norm.weight"] + p["norm.bias"]
    return torch.nn.functional.cross_entropy(z.mean(1) @ p["embedding"].T, targets)


@pytest.mark.parametrize("dtype,tol,act", [(torch.float32, 1e-4, "silu"), (torch.float32, 1e-4, "gelu"),
                                           (torch.bfloat16, 1.2e-1, "silu")])
def test_gradients_match_autograd(dtype, tol, act):
    """fp32: the gradients' own 1e-4; bf16: two dozen roundings of 2^-9 in a row a layer, over two layers."""
    cfg = Config(vocab=50, d_model=64, layers=2, heads=2, d_head=64, rank=8, dtype=dtype, d_ff=136, activation=act)
    model = Decoder(cfg)
    g = torch.Generator().manual_seed(3)
    ids, targets = (torch.randint(0, 50, (150,), generator=g) for _ in range(2))
    starts = torch.tensor([0, 1, 131, 150])
    loss, grads = model.gradients(ids.cuda(), targets.cuda(), starts.int().cuda())
    p = {k: t.double().cpu().requires_grad_() for k, t in model.params.items()}
    want = plain_loss(cfg, p, model.log_decay.double().cpu(), ids, targets, starts)
    want.backward()
    assert abs(loss.item() - want.item()) <= tol * want.item()
    assert set(grads) == set(p)
    for k in p:
        ref = p[k].grad
        assert (grads[k].double().cpu() - ref).norm() <= tol * ref.norm(), k


@pytest.mark.parametrize("dtype,fp8,tol", [(torch.float32, False, 1e-4), (torch.bfloat16, False, 4e-2),
                                           (torch.bfloat16, True, 0.25)])
def test_steps_continue_a_prompt(dtype, fp8, tol):
    """FP8: a rounding that falls the other way moves a code by up to 2^-3 of its value, in each of x and h."""
    cfg = Config(vocab=100, d_model=256, layers=3, heads=2, d_head=64, rank=16, dtype=dtype, d_ff=640, fp8=fp8)
    model = Decoder(cfg, slots=5, seed=1)
    ids = torch.randint(0, 100, (2, 170), generator=torch.Generator().manual_seed(4)).cuda()
    both = torch.tensor([0, 170, 340], dtype=torch.int32, device="cuda")
    want = model.prompt(ids.flatten(), both).float().view(2, 170, -1)
    heads = torch.tensor([0, 133, 293], dtype=torch.int32, device="cuda")
    first = model.prompt(torch.cat([ids[0, :133], ids[1, :160]]), heads, torch.tensor([4, 1], device="cuda")).float()
    assert (first[:133] - want[0, :133]).norm() <= tol * want[0, :133].norm()
    for t in range(10):
        both_now = torch.stack([ids[0, 133 + t], ids[1, 160 + t]])
        got = model.step(both_now, torch.tensor([4, 1], dtype=torch.int32, device="cuda")).float()
        ref = torch.stack([want[0, 133 + t], want[1, 160 + t]])
        assert (got - ref).norm() <= tol * ref.norm(), t


def test_fp8_stays_near_bf16():
    """Four encodings a block (x, both weights, h), each off by at most 2^-4 of a value."""
    cfg = dict(vocab=100, d_model=256, layers=2, heads=2, d_head=64, rank=16, d_ff=512)
    ids = torch.randint(0, 100, (300,), generator=torch.Generator().manual_seed(5)).cuda()
    starts = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    a, b = (Decoder(Config(**cfg, fp8=fp8), seed=2).prompt(ids, starts).float() for fp8 in (False, True))
    assert 0 < (a - b).norm() <= 4 * 2.0 ** -4 * a.norm()


def test_without_feed_forward_the_parameters_are_as_before():
    plain, wide = Decoder(Config(), seed=7), Decoder(Config(d_ff=64), seed=7)
    assert set(plain.params) < set(wide.params)
    assert torch.equal(plain.params["embedding"], wide.params["embedding"])
    assert not any(".ff" in k for k in plain.params) and len(plain.packed) == plain.cfg.layers


def test_the_command_runs(capsys):
    decoder.main(["--d-ff", "256", "--fp8"])
    assert "continued 24 tokens" in capsys.readouterr().out
