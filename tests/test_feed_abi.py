"""The entries of the feed-forward sublayer and of FP8 blocks refuse bad arguments on the host, before any CUDA
call: with good ones this host (no GPU) answers GR_E_DEVICE, so every other status came from the checks."""
from __future__ import annotations

import ctypes
from ctypes import byref

import pytest
import torch

from stream_gated_residual_gb300 import build as gbuild
from stream_gated_residual_gb300 import gr
from test_abi import header_constant as E

NULL = ctypes.c_void_p(None)
BIG = 1 << 34    # apart from each other


def P(k, off=0):
    return ctypes.c_void_p(BIG * (k + 1) + off)


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    if torch.cuda.is_available():
        pytest.skip("the addresses below are made up: only for hosts without a GPU")
    return gr.load()


def feed(n=10, d=64, f=128, dtype=1, act=0):
    return gr.FeedStruct(n, d, f, dtype, act)


def size(lib, name, *args):
    n = ctypes.c_size_t(0)
    assert getattr(lib, name)(*args, byref(n)) == 0
    return n.value


BAD_FEED = [(dict(n=-1), "GR_E_SHAPE"), (dict(n=1 << 31), "GR_E_SHAPE"), (dict(d=0), "GR_E_SHAPE"), (dict(d=12), "GR_E_SHAPE"),
            (dict(d=12296), "GR_E_SHAPE"), (dict(f=4), "GR_E_SHAPE"), (dict(f=131080), "GR_E_SHAPE"),
            (dict(act=2), "GR_E_SHAPE"), (dict(act=-1), "GR_E_SHAPE"), (dict(dtype=3), "GR_E_DTYPE"),
            (dict(dtype=-1), "GR_E_DTYPE")]


@pytest.mark.parametrize("kw,code", BAD_FEED)
def test_feed_shapes(lib, kw, code):
    f, n = feed(**kw), ctypes.c_size_t(0)
    for gradient in (0, 1):
        assert lib.gr_feed_workspace_size(byref(f), gradient, byref(n)) == E(code)
    assert lib.gr_feed_forward(byref(f), P(0), P(1), P(2), P(3), P(4), P(5), 1 << 30, NULL) == E(code)
    assert lib.gr_feed_forward_backward(byref(f), *map(P, range(9)), 1 << 30, NULL) == E(code)
    if "dtype" not in kw:
        f.dtype = 2
        assert lib.gr_feed_forward_fp8(byref(f), *map(P, range(7)), 1 << 30, NULL) == E(code)


def test_feed_dtypes(lib):
    """FP8 is the dtype of gr_feed_forward_fp8 alone, and has no gradient."""
    n = ctypes.c_size_t(0)
    f8, bf = feed(dtype=2), feed()
    assert lib.gr_feed_workspace_size(byref(f8), 0, byref(n)) == 0
    assert lib.gr_feed_workspace_size(byref(f8), 1, byref(n)) == E("GR_E_DTYPE")
    assert lib.gr_feed_forward(byref(f8), *map(P, range(6)), 1 << 30, NULL) == E("GR_E_DTYPE")
    assert lib.gr_feed_forward_fp8(byref(bf), *map(P, range(7)), 1 << 30, NULL) == E("GR_E_DTYPE")
    assert lib.gr_feed_workspace_size(byref(feed(d=72, dtype=2)), 0, byref(n)) == E("GR_E_SHAPE")
    assert lib.gr_feed_workspace_size(byref(feed(f=136, dtype=2)), 0, byref(n)) == E("GR_E_SHAPE")
    assert lib.gr_feed_workspace_size(None, 0, byref(n)) == E("GR_E_NULL")
    assert lib.gr_feed_workspace_size(byref(bf), 0, None) == E("GR_E_NULL")


@pytest.mark.parametrize("dtype", [0, 1])
def test_feed_forward_arguments(lib, dtype):
    f = feed(dtype=dtype)
    w = (4, 2)[dtype]
    need = size(lib, "gr_feed_workspace_size", byref(f), 0)
    good = dict(x=P(0), wi=P(1), wo=P(2), y=P(3), pre=P(4), ws=P(5), n=need)
    call = lambda **kw: lib.gr_feed_forward(byref(f), *{**good, **kw}.values(), NULL)  # noqa: E731
    assert call() == E("GR_E_DEVICE")
    assert call(pre=NULL) == E("GR_E_DEVICE")
    for k in ("x", "wi", "wo", "y"):
        assert call(**{k: NULL}) == E("GR_E_NULL")
    for i, k in enumerate(("x", "wi", "wo", "y", "pre")):
        assert call(**{k: P(i, 8)}) == E("GR_E_ALIGN")
    assert call(n=need - 1) == E("GR_E_SIZE") == call(ws=NULL)
    assert call(ws=P(5, 128)) == E("GR_E_ALIGN")
    for bad in (dict(y=P(0)), dict(y=P(1, 2 * 128 * 64 * w - 16)), dict(y=P(2)), dict(y=P(4, 16)), dict(pre=P(0)),
                dict(pre=P(3)), dict(ws=P(0)), dict(ws=P(1)), dict(ws=P(2)), dict(ws=P(3)), dict(y=P(5, need - 256))):
        assert call(**bad) == E("GR_E_ALIAS"), bad
    assert lib.gr_feed_forward(None, *good.values(), NULL) == E("GR_E_NULL")
    empty = feed(n=0, dtype=dtype)
    assert lib.gr_feed_forward(byref(empty), *[NULL] * 6, 0, NULL) == 0


@pytest.mark.parametrize("dtype", [0, 1])
def test_feed_backward_arguments(lib, dtype):
    f = feed(dtype=dtype)
    need = size(lib, "gr_feed_workspace_size", byref(f), 1)
    names = ("dy", "x", "wi", "wo", "pre", "dx", "dwi", "dwo", "ws")
    good = {**{k: P(i) for i, k in enumerate(names)}, "n": need}
    call = lambda **kw: lib.gr_feed_forward_backward(byref(f), *{**good, **kw}.values(), NULL)  # noqa: E731
    assert call() == E("GR_E_DEVICE")
    for i, k in enumerate(names[:8]):
        assert call(**{k: NULL}) == E("GR_E_NULL")
        assert call(**{k: P(i, 4)}) == E("GR_E_ALIGN")
    assert call(n=need - 1) == E("GR_E_SIZE") == call(ws=NULL)
    assert call(ws=P(8, 16)) == E("GR_E_ALIGN")
    for out in ("dx", "dwi", "dwo"):
        for i in range(9):
            if names[i] != out:
                assert call(**{out: P(i)}) == E("GR_E_ALIAS"), (out, names[i])
    for i in range(5):
        assert call(ws=P(i)) == E("GR_E_ALIAS")
    # no tokens: the weights' gradients are still written
    empty = feed(n=0, dtype=dtype)
    assert lib.gr_feed_forward_backward(byref(empty), *[NULL] * 5, NULL, P(6), P(7), NULL, 0, NULL) == E("GR_E_DEVICE")
    assert lib.gr_feed_forward_backward(byref(empty), *[NULL] * 5, NULL, NULL, P(7), NULL, 0, NULL) == E("GR_E_NULL")


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), "GR_E_SHAPE"), (dict(cols=24), "GR_E_SHAPE"), (dict(cols=0), "GR_E_SHAPE"),
    (dict(cols=131088), "GR_E_SHAPE"), (dict(nm=0), "GR_E_SHAPE"), (dict(br=64), "GR_E_SHAPE"), (dict(dtype=2), "GR_E_DTYPE"),
    (dict(rows=1 << 31, cols=16), "GR_E_SHAPE"), (dict(rows=1 << 30, cols=272), "GR_E_SHAPE"),
    (dict(rows=1 << 62, nm=1 << 30), "GR_E_SHAPE")])
def test_blocks_shapes(lib, kw, code):
    a = dict(rows=10, cols=256, nm=1, br=1, dtype=1, **{}) | kw
    b = gr.BlocksStruct(a["rows"], a["cols"], a["nm"], a["br"], a["dtype"])
    assert lib.gr_fp8_encode_blocks(byref(b), P(0), P(1), P(2), NULL) == E(code)


def test_blocks_arguments(lib):
    b = gr.BlocksStruct(10, 272, 2, 1, 1)
    call = lambda m=P(0), c=P(1), s=P(2): lib.gr_fp8_encode_blocks(byref(b), m, c, s, NULL)  # noqa: E731
    assert call() == E("GR_E_DEVICE") == call(s=P(2, 3))
    for bad in (dict(m=NULL), dict(c=NULL), dict(s=NULL)):
        assert call(**bad) == E("GR_E_NULL")
    for bad in (dict(m=P(0, 8)), dict(c=P(1, 4))):
        assert call(**bad) == E("GR_E_ALIGN")
    for bad in (dict(c=P(0)), dict(s=P(0, 20 * 272 * 2 - 1)), dict(s=P(1, 20 * 272 - 1))):
        assert call(**bad) == E("GR_E_ALIAS")
    assert lib.gr_fp8_encode_blocks(None, P(0), P(1), P(2), NULL) == E("GR_E_NULL")
    assert lib.gr_fp8_encode_blocks(byref(gr.BlocksStruct(0, 272, 2, 1, 1)), NULL, NULL, NULL, NULL) == 0


@pytest.mark.parametrize("n,k,o", [(-1, 64, 64), (1 << 31, 64, 64), (4, 24, 64), (4, 0, 64), (4, 131088, 64), (4, 64, 4),
                                   (4, 64, 262152)])
def test_product_shapes(lib, n, k, o):
    p, m = gr.ProductStruct(n, k, o), ctypes.c_size_t(0)
    assert lib.gr_fp8_matmul_workspace_size(byref(p), byref(m)) == E("GR_E_SHAPE")
    assert lib.gr_fp8_matmul(byref(p), *map(P, range(6)), 1 << 30, NULL) == E("GR_E_SHAPE")


def test_product_arguments(lib):
    p = gr.ProductStruct(10, 272, 136)
    need = size(lib, "gr_fp8_matmul_workspace_size", byref(p))
    names = ("a", "as_", "b", "bs", "out", "ws")
    good = {**{k: P(i) for i, k in enumerate(names)}, "n": need}
    call = lambda **kw: lib.gr_fp8_matmul(byref(p), *{**good, **kw}.values(), NULL)  # noqa: E731
    assert call() == E("GR_E_DEVICE") == call(as_=P(1, 1), bs=P(3, 3))
    for i, k in enumerate(names[:5]):
        assert call(**{k: NULL}) == E("GR_E_NULL")
    for k, i in (("a", 0), ("b", 2), ("out", 4)):
        assert call(**{k: P(i, 8)}) == E("GR_E_ALIGN")
    assert call(n=need - 1) == E("GR_E_SIZE") == call(ws=NULL)
    for i in range(4):
        assert call(out=P(i)) == E("GR_E_ALIAS") == call(ws=P(i))
    assert call(out=P(5)) == E("GR_E_ALIAS")
    assert lib.gr_fp8_matmul(byref(gr.ProductStruct(0, 272, 136)), *[NULL] * 6, 0, NULL) == 0


def test_feed_fp8_arguments(lib):
    f = feed(dtype=2)
    need = size(lib, "gr_feed_workspace_size", byref(f), 0)
    names = ("x", "wi", "wis", "wo", "wos", "y", "ws")
    good = {**{k: P(i) for i, k in enumerate(names)}, "n": need}
    call = lambda **kw: lib.gr_feed_forward_fp8(byref(f), *{**good, **kw}.values(), NULL)  # noqa: E731
    assert call() == E("GR_E_DEVICE") == call(wis=P(2, 1))
    for k in names[:6]:
        assert call(**{k: NULL}) == E("GR_E_NULL")
    assert call(n=need - 1) == E("GR_E_SIZE") == call(ws=NULL)
    for i in range(5):
        assert call(y=P(i)) == E("GR_E_ALIAS") == call(ws=P(i))
    assert lib.gr_feed_forward_fp8(byref(feed(n=0, dtype=2)), *[NULL] * 7, 0, NULL) == 0


@pytest.mark.parametrize("dtype,gradient", [(0, 0), (0, 1), (1, 0), (1, 1), (2, 0)])
def test_workspaces_grow_with_the_call(lib, dtype, gradient):
    """Every size from one token to many has a workspace that holds the hidden values at least; what passes any
    memory is planned or refused."""
    n = ctypes.c_size_t(0)
    for tokens in (0, 1, 7, 64, 256, 257, 512, 513, 4096, 100_003, (1 << 31) - 1):
        for d, f in ((16, 16), (2560, 10240), (12288, 131072)):
            status = lib.gr_feed_workspace_size(byref(feed(tokens, d, f, dtype)), gradient, byref(n))
            if tokens < 1 << 30:
                assert status == 0
            assert status == E("GR_E_SHAPE") or status == 0 and n.value >= tokens * f * (1, 2)[dtype != 2], (tokens, d, f)
    for tokens in (0, 1, 600, (1 << 31) - 1):
        for k, o in ((16, 8), (131072, 262144)):
            p = gr.ProductStruct(tokens, k, o)
            assert lib.gr_fp8_matmul_workspace_size(byref(p), byref(n)) in (0, E("GR_E_SHAPE"))
