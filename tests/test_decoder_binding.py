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
    monkeypatch.setattr(gr, "_several_devices", lambda: True)
    monkeypatch.setattr(gr, "_current_device", lambda: -1)   # where CPU tensors are
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


class Launches:
    """The library with its launching entries answering 0."""

    def __init__(self, lib):
        self.lib = lib

    def __getattr__(self, name):
        return getattr(self.lib, name) if name.endswith("_size") else lambda *args: 0


@pytest.mark.parametrize("name", ["pack_params", "read", "read large rank", "write_then_read", "read_fixed_gates",
                                  "read_backward", "write_backward", "decompose", "fp8_encode", "fp8_decode", "read_fp8",
                                  "write_then_read_fp8"])
def test_residual_outputs_are_recorded_on_the_stream(calls, monkeypatch, name):
    """The same for the reads and writes, and for the workspaces that a call makes and drops itself."""
    lib = Launches(gr.load())
    monkeypatch.setattr(gr, "load", lambda: lib)
    stream, made, empty = Stream(), [], torch.empty
    N, D, r = 3, 64, 4
    F, B = torch.float32, torch.bfloat16
    rank = 320 if name == "read large rank" else r
    if rank > r:
        N, D = 5, 2560
    R, y, s = torch.zeros(N, 4, D, dtype=B), torch.zeros(N, D, dtype=B), torch.zeros(N, 4)
    weights = torch.ones(4, D), torch.zeros(r, 4 * D), torch.zeros(4 * D, r), torch.zeros(4, 4 * D)
    fp8 = torch.zeros(N, 4, D, dtype=torch.uint8), torch.zeros(N, 4, D // 32, dtype=torch.uint8)
    params = gr.Params(torch.zeros(1), gr.ParamsStruct(None, D, 4, rank, gr.GR_BF16, gr.GR_PARAMS_TAG), B, 1e-6)

    def counted(*args, **kw):
        made.append(empty(*args, **kw))
        return made[-1]

    def counted_like(t, **kw):
        return counted(t.shape, dtype=t.dtype, device=t.device)

    run = {
        "pack_params": lambda: gr.pack_params(*weights, B, stream=stream),
        "read": lambda: gr.read(R, params, stream=stream),
        "read large rank": lambda: gr.read(R, params, stream=stream),
        "write_then_read": lambda: gr.write_then_read(R, y, s, params, stream=stream),
        "read_fixed_gates": lambda: gr.read_fixed_gates(R, weights[0], R, stream=stream),
        "read_backward": lambda: gr.read_backward(R, *weights, torch.zeros(N, D), s, stream=stream),
        "write_backward": lambda: gr.write_backward(R.float(), y, s, stream=stream),
        "decompose": lambda: gr.decompose(R, *weights, y[None], s[None], R, stream=stream),
        "fp8_encode": lambda: gr.fp8_encode(R, stream=stream),
        "fp8_decode": lambda: gr.fp8_decode(*fp8, stream=stream),
        "read_fp8": lambda: gr.read_fp8(*fp8, params, stream=stream),
        "write_then_read_fp8": lambda: gr.write_then_read_fp8(*fp8, y, s, params, stream=stream),
    }[name]
    monkeypatch.setattr(torch, "empty", counted)
    monkeypatch.setattr(torch, "empty_like", counted_like)
    run()
    got = {p for p, on in calls.recorded if on is stream}
    assert made and all(t.data_ptr() in got for t in made)


@pytest.mark.parametrize("i", range(7))
def test_tensors_of_another_device_are_refused(calls, monkeypatch, i):
    """Every launch goes to the current device: a tensor of another one is a ValueError, whichever argument it is."""
    monkeypatch.setattr(gr, "_current_device", lambda: 1)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1, raising=False)
    name, call = operators(Stream())[i]
    made, new = [], gr._new
    monkeypatch.setattr(gr, "_new", lambda *a: made.append(new(*a)) or made[-1])
    call()
    assert len(calls) == 1
    pointers = [struct.unpack("=Q", a[:8])[0] if isinstance(a, bytes) and len(a) == 24 else a
                for a in calls[0][1][1:]]
    arguments = {p for p in pointers if isinstance(p, int) and p > 1 << 20 and p != STREAM}
    arguments -= {t.data_ptr() for t in made}           # which are made on the first tensor's device
    asked = []
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: asked.append(t.data_ptr()) or 1, raising=False)
    call()
    assert len(asked) >= len(arguments), name           # every tensor whose address goes to the library was asked
    for at in range(len(asked)):
        count = iter(range(1000))
        monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0 if next(count) == at else 1, raising=False)
        before = len(calls)
        with pytest.raises(ValueError, match="device"):
            call()
        assert len(calls) == before
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0, raising=False)
    with pytest.raises(ValueError, match="device"):     # all on one device, another one than the current
        call()


def test_descriptors_hold_values_not_tensors(calls):
    """A scale or eps given as a tensor counts at its value of the call, also when it changed since the last one."""
    D, N, H, d = 16, 4, 1, 64
    ids, w, x = torch.zeros(N, dtype=torch.int64), torch.ones(4, D), torch.zeros(N, 4, D)
    q, decay, state = torch.zeros(N, H, d), torch.zeros(H), torch.zeros(N, H, d, d)
    s, at = torch.tensor(0.5), torch.zeros(5, D)
    forms = [lambda: gr.embed(at, ids, s, stream=Stream()), lambda: gr.embed_backward(x, ids, 5, s, stream=Stream()),
             lambda: gr.layer_norm(x, w, None, s, stream=Stream()),
             lambda: gr.linear_attention(q, q, q, decay, s, stream=Stream()),
             lambda: gr.linear_attention_step(q, q, q, decay, state, s, stream=Stream()),
             lambda: gr.linear_attention_backward(q, q, q, q, decay, s, stream=Stream())]
    for form in forms:
        for value in (0.5, 0.25):
            s.fill_(value)
            form()
            assert struct.unpack("=f", calls[-1][1][0][-4:])[0] == value, calls[-1][0]


def test_state_gradient_in_place(calls):
    """dstate_in is the caller's where it is given, dstate itself among them."""
    q, decay, ds = torch.zeros(3, 1, 64), torch.zeros(1), torch.zeros(1, 1, 64, 64)
    got = gr.linear_attention_backward(q, q, q, q, decay, dstate=ds, dstate_in=ds, stream=Stream())
    args = calls[-1][1]
    assert got[3] is ds and args[8] == ds.data_ptr() == args[12]
    alone = torch.zeros_like(ds)                        # also with neither state nor dstate
    got = gr.linear_attention_backward(q, q, q, q, decay, dstate_in=alone, stream=Stream())
    assert got[3] is alone and calls[-1][1][8] is None and calls[-1][1][12] == alone.data_ptr()
    for bad in (torch.zeros(1, 1, 64, 32), ds.to(torch.bfloat16), ds.transpose(2, 3)):
        with pytest.raises(ValueError, match="dstate_in"):
            gr.linear_attention_backward(q, q, q, q, decay, dstate_in=bad)


def test_embedding_workspace_is_what_the_plan_uses():
    """Two partial rows a piece of the largest tile: pieces of 64 sorted positions once they fill the SMs (four
    of a piece's columns an SM), 4 at least; twice that and the sort's 8 bytes a token cover any plan."""
    gbuild.build()
    for D in (8, 512, 520, 1024, 2560, 4096, 12288):
        cols = -(-D // 512)
        for N in (1, 3, 4, 777, 1024, 4096, 10000, 16383, 16384, 16385, 100000, 1 << 24):
            tile = min(N, 16384)
            fill = 2 * (4 * 152) // cols + 1            # pieces that a halved piece can still reach
            pieces = min(-(-tile // 4), max(-(-tile // 64), fill))
            e = gr._embed_desc(N, 1000, D, 4, gr.GR_F32, gr.GR_F32, 64, 1.0)
            need = gr._need("gr_embed_backward_workspace_size", e)
            assert need <= 8 * N + 2 * 2 * pieces * D * 4 + 1024, (N, D)
            assert need >= 8 * N + 2 * -(-tile // 64) * D * 4
