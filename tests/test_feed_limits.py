"""Calls that are too large for the feed-forward kernels are refused on the host, before anything is launched."""
from __future__ import annotations

import ctypes
from ctypes import byref

import pytest

from stream_gated_residual_gb300 import build as gbuild
from stream_gated_residual_gb300 import gr
from test_abi import header_constant as E

FAR = 1 << 50    # made-up addresses, apart from each other; a refused call touches none of them


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gr.load()


@pytest.mark.parametrize("gradient", [0, 1])
@pytest.mark.parametrize("d,f", [(8, 8192), (8192, 8), (64, 131072)])
def test_fp32_calls_past_the_limit(lib, gradient, d, f):
    """N · max(D, F) is at most 2^34 - 1024: the last N that fits is planned, the next is refused by the size and by
    the call itself."""
    most = ((1 << 34) - 1024) // max(d, f)
    n = ctypes.c_size_t(0)
    assert lib.gr_feed_workspace_size(byref(gr.FeedStruct(most, d, f, 0, 0)), gradient, byref(n)) == 0
    assert n.value > 6 * most * f
    past = gr.FeedStruct(most + 1, d, f, 0, 0)
    assert lib.gr_feed_workspace_size(byref(past), gradient, byref(n)) == E("GR_E_SHAPE")
    p = [ctypes.c_void_p(FAR * (k + 1)) for k in range(9)]
    if gradient:
        assert lib.gr_feed_forward_backward(byref(past), *p, 1 << 48, None) == E("GR_E_SHAPE")
    else:
        assert lib.gr_feed_forward(byref(past), *p[:6], 1 << 48, None) == E("GR_E_SHAPE")


def test_bf16_has_no_such_limit(lib):
    n = ctypes.c_size_t(0)
    assert lib.gr_feed_workspace_size(byref(gr.FeedStruct(1 << 21, 8, 8200, 1, 0)), 0, byref(n)) == 0
