"""The binding's own part of the feed-forward calls, on the CPU (see test_decoder_binding for how)."""
from __future__ import annotations

import pytest
import torch

from stream_gated_residual_gb300 import gr
from test_decoder_binding import Stream, calls  # noqa: F401

N, D, F = 5, 64, 144


def operators(stream):
    B = torch.bfloat16
    x, w_in, w_out = torch.zeros(N, D, dtype=B), torch.zeros(2, F, D, dtype=B), torch.zeros(D, F, dtype=B)
    pre = torch.zeros(N, 2, F, dtype=B)

    def eight(rows, *shape):
        scales = (*shape[:-2], -(-shape[-2] // rows), -(-shape[-1] // 128))
        return torch.zeros(*shape, dtype=torch.uint8), torch.zeros(scales, dtype=torch.uint8)

    return [
        ("feed_forward", lambda: gr.feed_forward(x, w_in, w_out, keep=True, stream=stream)),
        ("feed_forward_backward", lambda: gr.feed_forward_backward(x, x, w_in, w_out, pre, stream=stream)),
        ("fp8_encode_blocks", lambda: gr.fp8_encode_blocks(x, stream=stream)),
        ("fp8_matmul", lambda: [gr.fp8_matmul(eight(1, N, D), eight(128, F, D), stream=stream)]),
        ("feed_forward_fp8", lambda: [gr.feed_forward_fp8(x, eight(128, 2, F, D), eight(128, D, F), stream=stream)]),
    ]


@pytest.mark.parametrize("i", range(5))
def test_outputs_and_workspaces_are_recorded_on_the_stream(calls, monkeypatch, i):  # noqa: F811
    made, empty = [], torch.empty

    def counted(*args, **kw):
        made.append(empty(*args, **kw))
        return made[-1]

    stream = Stream()
    name, call = operators(stream)[i]
    monkeypatch.setattr(torch, "empty", counted)
    outs = call()
    got = {p for p, on in calls.recorded if on is stream}
    assert {t.data_ptr() for t in outs} <= got and all(t.data_ptr() in got for t in made), name
    assert calls[-1][0] == "gr_" + name and calls[-1][1][-1] == stream.cuda_stream


@pytest.mark.parametrize("i", range(5))
def test_tensors_of_another_device_are_refused(calls, monkeypatch, i):  # noqa: F811
    name, call = operators(Stream())[i]
    call()
    monkeypatch.setattr(gr, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="device"):
        call()


def test_plans_are_kept_by_shape_and_not_by_tensor(calls):  # noqa: F811
    """The same call on tensors of another size gets another descriptor and workspace."""
    B = torch.bfloat16
    sizes = []
    for n in (3, 700, 3):
        gr.feed_forward(torch.zeros(n, D, dtype=B), torch.zeros(2, F, D, dtype=B), torch.zeros(D, F, dtype=B),
                        stream=Stream())
        args = calls[-1][1]
        sizes.append((args[0], args[7]))
    assert sizes[0] == sizes[2] != sizes[1]


@pytest.mark.parametrize("bad", [
    dict(x=torch.zeros(N, D)), dict(w_in=torch.zeros(F, D, dtype=torch.bfloat16)), dict(activation="tanh"),
    dict(w_out=torch.zeros(F, D, dtype=torch.bfloat16)), dict(y=torch.zeros(N, D)),
    dict(pre=torch.zeros(N, F, dtype=torch.bfloat16)), dict(x=torch.zeros(D, N, dtype=torch.bfloat16).T)])
def test_feed_forward_refuses(calls, bad):  # noqa: F811
    B = torch.bfloat16
    good = dict(x=torch.zeros(N, D, dtype=B), w_in=torch.zeros(2, F, D, dtype=B), w_out=torch.zeros(D, F, dtype=B))
    with pytest.raises(ValueError):
        gr.feed_forward(**{**good, **bad})
    assert not calls
