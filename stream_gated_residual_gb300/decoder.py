"""A small decoder on the library's calls: token embedding into the 4-branch state, a Gated Residual read, a
linear-attention mixer and a write per layer, the branches' layer norm, and tied logits.

    R = embed(E, ids)                        [N, 4, D]
    for each layer:  x, s = read(R);  y = W_o · linear_attention(W_qkv · x);  R += s_i y
    logits = E · mean_i layer_norm(R)_i

``prompt`` runs packed sequences and leaves each one's mixer states in a slot, ``step`` goes on one token a
request, ``gradients`` is a training step's forward and backward pass. The projections are plain
torch products; everything else is the library's. ``python -m stream_gated_residual_gb300.decoder``
trains one for a moment and lets it continue a prompt.

One read a layer, no MLP sublayer: the read, write and mixer are those of "【论文解读】 Qwen3.8 Flash Next"
(wkq9411.github.io), §二.4, with a plain linear attention in the place of its token mixer.
"""
from __future__ import annotations

import dataclasses
import math

import torch

from . import gr


@dataclasses.dataclass(frozen=True)
class Config:
    vocab: int = 512
    d_model: int = 256
    layers: int = 2
    heads: int = 4
    d_head: int = 64
    rank: int = 16
    dtype: torch.dtype = torch.bfloat16
    eps: float = 1e-6


class Decoder:
    def __init__(self, cfg: Config, slots: int = 0, seed: int = 0, device="cuda"):
        self.cfg = cfg
        g = torch.Generator(device="cpu")
        g.manual_seed(seed)
        D, K, H, r = cfg.d_model, 4 * cfg.d_model, cfg.heads * cfg.d_head, cfg.rank

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g) * std).to(device)

        self.params = {"embedding": normal(cfg.vocab, D, std=D ** -0.5),
                       "norm.weight": torch.ones(4, D, device=device),
                       "norm.bias": torch.zeros(4, D, device=device)}
        for i in range(cfg.layers):
            self.params.update({
                f"{i}.gamma": torch.ones(4, D, device=device),
                f"{i}.w_down": normal(r, K, std=0.02), f"{i}.w_up": normal(K, r, std=0.02),
                f"{i}.w_write": normal(4, K, std=0.02),
                f"{i}.qkv": normal(3 * H, D, std=D ** -0.5), f"{i}.out": normal(D, H, std=H ** -0.5)})
        # memories from a few tokens to a few hundred; constants of the model
        self.log_decay = -torch.exp2(-torch.linspace(1, 8, cfg.heads, device=device))
        # the requests' mixer states, a slot each: [layer][slot, head, d, d] fp32
        self.states = [torch.zeros(slots, cfg.heads, cfg.d_head, cfg.d_head, device=device)
                       for _ in range(cfg.layers)]
        self.pack()

    def pack(self) -> None:
        """The parameters in the forms the forward pass takes (after every update of ``params``)."""
        p, c = self.params, self.cfg
        self.packed = [gr.pack_params(p[f"{i}.gamma"], p[f"{i}.w_down"], p[f"{i}.w_up"], p[f"{i}.w_write"],
                                      c.dtype, c.eps) for i in range(c.layers)]
        self.cast = {k: p[k].to(c.dtype) for k in p if k == "embedding" or k.endswith((".qkv", ".out"))}

    def _embed(self, ids):
        return gr.embed(self.params["embedding"], ids, math.sqrt(self.cfg.d_model), dtype=self.cfg.dtype)

    def _qkv(self, i, x):
        c = self.cfg
        return (x @ self.cast[f"{i}.qkv"].T).view(-1, 3, c.heads, c.d_head).unbind(1)

    def _layers(self, R, mix, keep=None):
        """All layers on R in place; mix(i, q, k, v) -> o. `keep` collects what the gradients need."""
        x, s = gr.read(R, self.packed[0])
        for i in range(self.cfg.layers):
            q, k, v = self._qkv(i, x)
            o = mix(i, q, k, v)
            y = o.flatten(1) @ self.cast[f"{i}.out"].T
            if keep is not None:
                keep.append((R.clone(), x, s, q, k, v, o, y))
            if i + 1 < self.cfg.layers:
                x, s = gr.write_then_read(R, y, s, self.packed[i + 1])
            else:
                gr.write(R, y, s)
        return R

    def _logits(self, R):
        z = gr.layer_norm(R, self.params["norm.weight"], self.params["norm.bias"], self.cfg.eps)
        return z.mean(1) @ self.cast["embedding"].T

    def prompt(self, ids, seq_starts, slots=None):
        """Logits [N, V] of packed sequences (ids [N], seq_starts int32 [B + 1]). With `slots` (int64 [B])
        each sequence's mixer states are left in its slot."""
        def mix(i, q, k, v):
            o, state = gr.linear_attention(q, k, v, self.log_decay, seq_starts=seq_starts)
            if slots is not None:
                self.states[i][slots] = state
            return o
        return self._logits(self._layers(self._embed(ids), mix))

    def step(self, ids, slots):
        """Logits [n, V] after one token of each of n requests (slots int32 [n])."""
        def mix(i, q, k, v):
            return gr.linear_attention_step(q, k, v, self.log_decay, self.states[i], slots=slots)
        return self._logits(self._layers(self._embed(ids), mix))

    def gradients(self, ids, targets, seq_starts):
        """(mean cross entropy, gradients like ``params``) of packed sequences."""
        c, p, N = self.cfg, self.params, ids.numel()
        scale = math.sqrt(c.d_model)
        kept = []
        R = self._layers(self._embed(ids), lambda i, q, k, v: gr.linear_attention(
            q, k, v, self.log_decay, seq_starts=seq_starts)[0], kept)
        z, mean, rstd = gr.layer_norm(R, p["norm.weight"], p["norm.bias"], c.eps, stats=True)
        top = z.float().mean(1)
        logp = torch.log_softmax(top @ p["embedding"].T, -1)
        loss = -logp[torch.arange(N, device=ids.device), targets].mean()
        dlogits = torch.exp(logp)
        dlogits[torch.arange(N, device=ids.device), targets] -= 1
        dlogits /= N
        g = {}
        dz = (dlogits @ p["embedding"] / 4)[:, None].expand(-1, 4, -1).contiguous()
        dR, g["norm.weight"], g["norm.bias"] = gr.layer_norm_backward(dz, R, p["norm.weight"], mean, rstd)
        for i in reversed(range(c.layers)):
            Ri, x, s, q, k, v, o, y = kept[i]
            dR, dy, ds = gr.write_backward(dR, y, s)
            g[f"{i}.out"] = dy.T @ o.flatten(1).float()
            do = (dy @ p[f"{i}.out"]).view(N, c.heads, c.d_head).to(c.dtype)
            dqkv = torch.empty(N, 3, c.heads, c.d_head, dtype=c.dtype, device=ids.device)
            gr.linear_attention_backward(do, q, k, v, self.log_decay, seq_starts=seq_starts,
                                         out=dqkv.unbind(1))
            dqkv = dqkv.flatten(1).float()
            g[f"{i}.qkv"] = dqkv.T @ x.float()
            dread, gi = gr.read_backward(Ri, p[f"{i}.gamma"], p[f"{i}.w_down"], p[f"{i}.w_up"],
                                         p[f"{i}.w_write"], dqkv @ p[f"{i}.qkv"], ds, c.eps)
            dR += dread
            g.update({f"{i}.{name}": t for name, t in gi.items()})
        # the table is tied: its rows' gradient on top of the logits'
        g["embedding"] = gr.embed_backward(dR, ids, c.vocab, scale, dtable=(dlogits.T @ top).contiguous(),
                                           accumulate=True)
        return loss, g


def main() -> None:
    """Learns to continue a repeated phrase, then continues it token by token."""
    cfg = Config()
    model = Decoder(cfg, slots=4)
    phrase = torch.randint(0, cfg.vocab, (12,), generator=torch.Generator().manual_seed(1)).cuda()
    text = phrase.repeat(40)
    starts = torch.tensor([0, 100, 229, 479], dtype=torch.int32, device="cuda")
    moment = {k: torch.zeros_like(t) for k, t in model.params.items()}
    for i in range(60):
        loss, g = model.gradients(text[:479].contiguous(), text[1:480].contiguous(), starts)
        for k, t in model.params.items():
            moment[k].mul_(0.9).add_(g[k])
            t.add_(moment[k], alpha=-0.02 / float(moment[k].norm().clamp(min=1e-2)))
        model.pack()
        if i % 20 == 0 or i == 59:
            print(f"step {i:2d}: loss {loss.item():.3f}")
    logits = model.prompt(text[:50].contiguous(), torch.tensor([0, 50], dtype=torch.int32, device="cuda"),
                          torch.tensor([2], device="cuda"))
    slot, token, said = torch.tensor([2], dtype=torch.int32, device="cuda"), logits[-1:].argmax(-1), []
    for _ in range(24):
        said.append(int(token))
        token = model.step(token, slot).argmax(-1)
    right = sum(a == int(b) for a, b in zip(said, text[50:74]))
    print(f"continued 24 tokens, {right} as in the text")


if __name__ == "__main__":
    main()
