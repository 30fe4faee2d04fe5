"""Workspace sizes follow the current device, on the CPU: a library whose sizes differ from device to device, as they
do where devices have different numbers of SMs, and a record of what the calls are given."""
from __future__ import annotations

import pytest
import torch

from stream_gated_residual_gb300 import gr
from test_decoder_binding import Stream, calls  # noqa: F401
from test_feed_binding import operators as feed_operators
from test_decoder_binding import operators as decoder_operators


@pytest.mark.parametrize("which,i", [(feed_operators, i) for i in (0, 1, 3, 4)] + [(decoder_operators, i) for i in (1, 3, 4, 6)])
def test_a_call_gets_the_current_devices_workspace(calls, monkeypatch, request, which, i):  # noqa: F811
    """The same call on one device, on another and on the first again."""
    device, asked, recorded, extra = [-1], [], gr._call, {-1: 1 << 16, 1: 1 << 20}

    def call(name, *args):
        recorded(name, *args)
        if name.endswith("_workspace_size"):
            args[-1]._obj.value += extra[device[0]]
            asked.append((device[0], args[-1]._obj.value))

    made, empty = [], torch.empty

    def counted(*args, **kw):
        made.append(empty(*args, **kw))
        return made[-1]

    monkeypatch.setattr(gr, "_call", call)
    monkeypatch.setattr(gr, "_current_device", lambda: device[0])
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: device[0])
    for kept in (gr._need_on, gr._feed_plan, gr._product_plan, gr._feed_fp8_plan):
        kept.cache_clear()     # sizes of the library as it is
        request.addfinalizer(kept.cache_clear)
    name, operator = which(Stream())[i]
    monkeypatch.setattr(torch, "empty", counted)
    for d in (-1, 1, -1):
        device[0] = d
        made.clear()
        operator()
        need = dict(asked)[d]
        assert any(t.numel() * t.element_size() == need for t in made), (name, d)
