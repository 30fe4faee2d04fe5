"""The decoder example end to end: its gradients against torch autograd of the same model in 64 bits, and its
token-by-token form against its prompt form."""
from __future__ import annotations

import math

import pytest
import torch

from stream_gated_residual_gb300 import gr
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
    decay = torch.where(live, torch.exp(log_decay[:, None, None] * gap.clamp(min=0)), 0.0)   # [H, N, N]
    R = (math.sqrt(cfg.d_model) * p["embedding"][ids])[:, None].expand(-1, 4, -1)
    for i in range(cfg.layers):
        n = R * p[f"{i}.gamma"] / (R.square().mean(-1, keepdim=True) + cfg.eps).sqrt()
        v = n.flatten(1)
        hidden = torch.nn.functional.silu(v @ p[f"{i}.w_down"].T / 4)
        G = torch.sigmoid(hidden @ p[f"{i}.w_up"].T).view_as(n)
        x = (G * n).mean(1)
        s = 2 * torch.sigmoid(v @ p[f"{i}.w_write"].T / 4)
        q, k, u = (x @ p[f"{i}.qkv"].T).view(N, 3, H, d).unbind(1)
        scores = torch.einsum("nhd,mhd->hnm", q, k) * decay * d ** -0.5
        o = torch.einsum("hnm,mhd->nhd", scores, u)
        R = R + s[:, :, None] * (o.flatten(1) @ p[f"{i}.out"].T)[:, None]
    c = R - R.mean(-1, keepdim=True)
    z = c / (c.square().mean(-1, keepdim=True) + cfg.eps).sqrt() * p["norm.weight"] + p["norm.bias"]
    return torch.nn.functional.cross_entropy(z.mean(1) @ p["embedding"].T, targets)


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 6e-2)])
def test_gradients_match_autograd(dtype, tol):
    """fp32: the gradients' own 1e-4; bf16: a dozen roundings of 2^-9 in a row a layer, over two layers."""
    cfg = Config(vocab=50, d_model=64, layers=2, heads=2, d_head=64, rank=8, dtype=dtype)
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


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 4e-2)])
def test_steps_continue_a_prompt(dtype, tol):
    cfg = Config(vocab=100, d_model=256, layers=3, heads=2, d_head=64, rank=16, dtype=dtype)
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
