"""The binding's own part of the decoder operators' calls, on the CPU: the C entries that would launch are
replaced by a record of their arguments, and every tensor claims to be a CUDA tensor."""
from __future__ import annotations

import struct

import pytest
import torch

from stream_gated_residual_gb300 import build as gbuild
from stream_gated_residual_gb300 import gr

STREAM = 0x5eed


class Stream:
    cuda_stream = STREAM


@pytest.fixture()
def calls(monkeypatch):
    """The launching calls [(entry, arguments)]; tensors recorded on a stream are in calls.recorded."""
    gbuild.build()
    gr.load()

    class Calls(list):
        recorded: list = []

    seen, whole = Calls(), gr._call
    seen.recorded = []

    def call(name, *args):
        if name.endswith("_workspace_size"):
            return whole(name, *args)
        seen.append((name, args))

    monkeypatch.setattr(gr, "_call", call)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True), raising=False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: seen.recorded.append((t.data_ptr(), s)),
                        raising=False)
    return seen


def operators(stream):
    """Every call with outputs of its own: (name, a call that gives all of them)."""
    N, H, d, D, V = 5, 2, 64, 16, 7
    ids, w = torch.zeros(N, dtype=torch.int64), torch.ones(4, D)
    x, st = torch.zeros(N, 4, D), torch.ones(N, 4)
    q = torch.zeros(N, H, d)
    state, decay = torch.zeros(1, H, d, d), torch.zeros(H)
    return [
        ("embed", lambda: [gr.embed(torch.zeros(V, D), ids, stream=stream)]),
        ("embed_backward", lambda: [gr.embed_backward(x, ids, V, stream=stream)]),
        ("layer_norm", lambda: gr.layer_norm(x, w, stats=True, stream=stream)),
        ("layer_norm_backward", lambda: gr.layer_norm_backward(x, x, w, st, st, stream=stream)),
        ("linear_attention", lambda: gr.linear_attention(q, q, q, decay, state=state, stream=stream)),
        ("linear_attention_step", lambda: [gr.linear_attention_step(q, q, q, decay, torch.zeros(N, H, d, d),
                                                                    stream=stream)]),
        ("linear_attention_backward", lambda: gr.linear_attention_backward(q, q, q, q, decay, state=state,
                                                                           stream=stream)),
    ]


@pytest.mark.parametrize("i", range(7))
def test_outputs_are_recorded_on_the_stream_that_writes_them(calls, i):
    """What a call makes comes from the current stream's memory: without the record, an output that is dropped
    early would be handed out again while `stream` still writes it."""
    stream = Stream()
    name, call = operators(stream)[i]
    made = [t.data_ptr() for t in call()]
    assert {p for p, s in calls.recorded if s is stream} >= set(made), name
