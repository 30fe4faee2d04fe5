"""The decoder operators' entries refuse bad arguments on the host, before any CUDA call: with good
ones this host (no GPU) answers GR_E_DEVICE, so every other status below came from the checks."""
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


def emb(n=10, v=100, d=64, nb=4, td=0, sd=1, bits=64, scale=1.0):
    return gr.EmbeddingStruct(n, v, d, nb, td, sd, bits, scale)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), "GR_E_SHAPE"), (dict(v=0), "GR_E_SHAPE"), (dict(v=1 << 31), "GR_E_SHAPE"), (dict(d=12), "GR_E_SHAPE"),
    (dict(d=12296), "GR_E_SHAPE"), (dict(nb=2), "GR_E_SHAPE"), (dict(td=2), "GR_E_DTYPE"), (dict(sd=7), "GR_E_DTYPE"),
    (dict(bits=16), "GR_E_DTYPE")])
def test_embedding_shapes(lib, kw, code):
    n = ctypes.c_size_t(0)
    assert lib.gr_embed(byref(emb(**kw)), P(0), P(1), P(2), NULL) == E(code)
    assert lib.gr_embed_backward_workspace_size(byref(emb(**kw)), byref(n)) == E(code)
    assert lib.gr_embed_backward(byref(emb(**kw)), P(0), P(1), P(2), 0, P(3), 1 << 30, NULL) == E(code)


def test_embedding_arguments(lib):
    e = emb()
    call = lambda t=P(0), i=P(1), r=P(2): lib.gr_embed(byref(e), t, i, r, NULL)  # noqa: E731
    assert call() == E("GR_E_DEVICE")
    assert call(i=P(1, 8)) == E("GR_E_DEVICE")                    # ids: natural alignment
    for bad in (dict(t=NULL), dict(i=NULL), dict(r=NULL)):
        assert call(**bad) == E("GR_E_NULL")
    for bad in (dict(t=P(0, 8)), dict(i=P(1, 4)), dict(r=P(2, 2))):
        assert call(**bad) == E("GR_E_ALIGN")
    assert call(r=P(0, 64 * 4 * 99)) == E("GR_E_ALIAS")
    assert lib.gr_embed(None, P(0), P(1), P(2), NULL) == E("GR_E_NULL")
    assert lib.gr_embed(byref(emb(n=0)), NULL, NULL, NULL, NULL) == 0
    n = ctypes.c_size_t(0)
    assert lib.gr_embed_backward_workspace_size(byref(e), byref(n)) == 0 and n.value >= 80
    back = lambda r=P(0), i=P(1), t=P(2), w=P(3), b=n.value: lib.gr_embed_backward(  # noqa: E731
        byref(e), r, i, t, 0, w, b, NULL)
    assert back() == E("GR_E_DEVICE")
    assert back(b=n.value - 1) == E("GR_E_SIZE")
    assert back(w=P(3, 16)) == E("GR_E_ALIGN")
    assert back(w=P(2, 256)) == E("GR_E_ALIAS") and back(t=P(0)) == E("GR_E_ALIAS")
    for bad in (dict(r=NULL), dict(i=NULL), dict(t=NULL), dict(w=NULL)):
        assert back(**bad) == E("GR_E_NULL")
    assert lib.gr_embed_backward(byref(emb(n=0)), NULL, NULL, P(0), 1, NULL, 0, NULL) == 0


def norm(n=10, d=64, g=4, dt=1, eps=1e-5):
    return gr.NormStruct(n, d, g, dt, eps)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), "GR_E_SHAPE"), (dict(d=4), "GR_E_SHAPE"), (dict(d=12296), "GR_E_SHAPE"), (dict(g=3), "GR_E_SHAPE"),
    (dict(dt=2), "GR_E_DTYPE"), (dict(eps=-1.0), "GR_E_EPS"), (dict(eps=float("nan")), "GR_E_EPS")])
def test_norm_shapes(lib, kw, code):
    n = ctypes.c_size_t(0)
    assert lib.gr_layer_norm(byref(norm(**kw)), *[P(i) for i in range(6)], NULL) == E(code)
    assert lib.gr_layer_norm_backward_workspace_size(byref(norm(**kw)), byref(n)) == E(code)
    assert lib.gr_layer_norm_backward(byref(norm(**kw)), *[P(i) for i in range(9)], 1 << 30, NULL) == E(code)


def test_norm_arguments(lib):
    d = norm()
    p = [P(i) for i in range(6)]              # x, weight, bias, y, mean, rstd

    def call(**at):
        q = list(p)
        for k, v in at.items():
            q[int(k[1:])] = v
        return lib.gr_layer_norm(byref(d), *q, NULL)

    assert call() == call(_2=NULL, _4=NULL, _5=NULL) == call(_3=P(0)) == E("GR_E_DEVICE")
    for i in (0, 1, 3):
        assert call(**{f"_{i}": NULL}) == E("GR_E_NULL")
    for i in (0, 1, 2, 3):
        assert call(**{f"_{i}": P(i, 8)}) == E("GR_E_ALIGN")
    assert call(_4=P(4, 2)) == E("GR_E_ALIGN")
    assert call(_3=P(0, 16)) == call(_3=P(1)) == call(_4=P(3)) == call(_5=P(4)) == E("GR_E_ALIAS")
    assert lib.gr_layer_norm(byref(norm(n=0)), *[NULL] * 7) == 0
    n = ctypes.c_size_t(0)
    assert lib.gr_layer_norm_backward_workspace_size(byref(d), byref(n)) == 0
    p = [P(i) for i in range(9)]              # dy, x, weight, mean, rstd, dx, dweight, dbias, workspace

    def back(b=n.value, **at):
        q = list(p)
        for k, v in at.items():
            q[int(k[1:])] = v
        return lib.gr_layer_norm_backward(byref(d), *q, b, NULL)

    assert back() == back(_7=NULL) == back(_5=P(0)) == E("GR_E_DEVICE")
    for i in (0, 1, 2, 3, 4, 5, 6, 8):
        assert back(**{f"_{i}": NULL}) == E("GR_E_NULL")
    assert back(b=n.value - 1) == E("GR_E_SIZE")
    assert back(_8=P(8, 16)) == back(_0=P(0, 4)) == E("GR_E_ALIGN")
    assert back(_6=P(7)) == back(_8=P(1, 256)) == back(_5=P(1)) == E("GR_E_ALIAS")


def mixer(n=20, b=2, h=3, dk=64, dv=64, dt=1, scale=1.0):
    return gr.MixerStruct(n, b, h, dk, dv, dt, scale)


def rows(k, ts=192, hs=64, off=0):
    return gr.RowsStruct(BIG * (k + 1) + off, ts, hs)


MIX_BAD = [(dict(n=-1), "GR_E_SHAPE"), (dict(n=1 << 31), "GR_E_SHAPE"), (dict(b=-1), "GR_E_SHAPE"), (dict(h=0), "GR_E_SHAPE"),
           (dict(b=1 << 20, h=1 << 12), "GR_E_SHAPE"), (dict(dk=12), "GR_E_SHAPE"), (dict(dv=264), "GR_E_SHAPE"),
           (dict(dt=2), "GR_E_DTYPE")]


@pytest.mark.parametrize("kw,code", MIX_BAD)
def test_mixer_shapes(lib, kw, code):
    n = ctypes.c_size_t(0)
    m = mixer(**kw)
    r = [byref(rows(i)) for i in range(7)]
    assert lib.gr_mixer_path(byref(m)) == b"invalid"
    assert lib.gr_linear_attention_workspace_size(byref(m), 0, byref(n)) == E(code)
    assert lib.gr_linear_attention(byref(m), *r[:3], P(8), P(9), NULL, r[3], NULL, P(10), 1 << 33, NULL) == E(code)
    assert lib.gr_linear_attention_step(byref(m), *r[:3], P(8), P(9), 4, NULL, r[3], NULL) == E(code)
    assert lib.gr_linear_attention_backward(byref(m), *r[:4], P(8), P(9), NULL, NULL, *r[4:], NULL, P(10), 1 << 33,
                                            NULL) == E(code)


def test_mixer_paths(lib):
    path = lambda **kw: lib.gr_mixer_path(byref(mixer(**kw)))  # noqa: E731
    assert path() == path(dk=128, dv=64) == path(dk=128, dv=128) == b"mixer_tc"
    assert path(dk=72) == path(dt=0) == path(dk=256) == b"mixer_simt"


def test_mixer_arguments(lib):
    m = mixer()
    need = ctypes.c_size_t(0)
    assert lib.gr_linear_attention_workspace_size(byref(m), 0, byref(need)) == 0
    good = dict(q=rows(0), k=rows(1), v=rows(2), o=rows(3), d=P(4), s=P(5), si=P(6), so=P(7), w=P(8), b=need.value, m=m)

    def call(**kw):
        a = dict(good, **kw)
        r = {x: byref(a[x]) if a[x] is not None else None for x in "qkvo"}
        return lib.gr_linear_attention(byref(a["m"]), r["q"], r["k"], r["v"], a["d"], a["s"], a["si"], r["o"], a["so"],
                                       a["w"], a["b"], NULL)

    assert call() == call(so=P(6)) == call(si=NULL) == call(so=NULL) == E("GR_E_DEVICE")
    for x in "qkvo":
        assert call(**{x: None}) == call(**{x: gr.RowsStruct(None, 192, 64)}) == E("GR_E_NULL")
        assert call(**{x: rows(3 if x == "o" else 0, off=8)}) == E("GR_E_ALIGN")
        assert call(**{x: rows(9, ts=196)}) == E("GR_E_ALIGN")
        assert call(**{x: rows(9, ts=32)}) == call(**{x: rows(9, hs=0)}) == call(**{x: rows(9, ts=-192)}) == E("GR_E_SHAPE")
        assert call(**{x: rows(9, ts=1 << 45)}) == E("GR_E_SHAPE")
    assert call(o=rows(3, ts=128)) == E("GR_E_SHAPE")                # its rows overlap
    assert call(d=NULL) == call(s=NULL) == E("GR_E_NULL")
    assert call(s=P(5, 2)) == call(si=P(6, 4)) == call(d=P(4, 1)) == E("GR_E_ALIGN")
    assert call(o=rows(0)) == call(so=P(0)) == call(so=P(6, 64)) == call(so=P(3)) == E("GR_E_ALIAS")
    # between the rows of a fused projection: allowed; on them: not
    wide = dict(q=rows(0, 1024), k=rows(0, 1024, off=384), v=rows(0, 1024, off=768))
    assert call(**wide, o=rows(0, 1024, off=1152)) == E("GR_E_DEVICE")
    assert call(**wide, o=rows(0, 1024, off=1024)) == E("GR_E_ALIAS")
    assert call(**wide, o=rows(0, 1024, off=1152 + 640)) == E("GR_E_ALIAS")
    # head-major rows; strides of dimensions of one are not looked at
    assert call(o=rows(3, ts=64, hs=64 * 20)) == E("GR_E_DEVICE")
    assert call(m=mixer(n=1, b=2, h=1), o=rows(3, ts=0, hs=0)) == E("GR_E_DEVICE")
    assert call(m=mixer(b=1), s=NULL) == E("GR_E_DEVICE")
    assert lib.gr_linear_attention(byref(mixer(b=0)), *[None] * 3, NULL, NULL, NULL, None, NULL, NULL, 0, NULL) == 0
    if need.value:
        assert call(b=need.value - 1) == call(w=NULL) == E("GR_E_SIZE")
        assert call(w=P(8, 16)) == E("GR_E_ALIGN")
        assert call(w=P(0)) == call(w=P(7)) == E("GR_E_ALIAS")


def test_mixer_step_arguments(lib):
    m = mixer()
    good = dict(q=rows(0), k=rows(1), v=rows(2), o=rows(3), d=P(4), st=P(5), n=30, sl=P(6))

    def call(**kw):
        a = dict(good, **kw)
        return lib.gr_linear_attention_step(byref(m), byref(a["q"]), byref(a["k"]), byref(a["v"]), a["d"], a["st"],
                                            a["n"], a["sl"], byref(a["o"]), NULL)

    assert call() == call(sl=NULL) == E("GR_E_DEVICE")
    assert call(n=-1) == E("GR_E_SHAPE")
    assert call(st=NULL) == call(d=NULL) == E("GR_E_NULL")
    assert call(st=P(5, 8)) == call(sl=P(6, 2)) == call(q=rows(0, off=2)) == E("GR_E_ALIGN")
    assert call(o=rows(5)) == call(o=rows(1)) == call(st=P(2)) == call(st=P(6)) == E("GR_E_ALIAS")


def test_mixer_backward_arguments(lib):
    m = mixer()
    need = ctypes.c_size_t(0)
    assert lib.gr_linear_attention_workspace_size(byref(m), 1, byref(need)) == 0
    names = ["do", "q", "k", "v", "dq", "dk", "dv"]
    good = {x: rows(i) for i, x in enumerate(names)}
    good.update(d=P(7), s=P(8), si=P(9), dso=P(10), dsi=P(11), w=P(12), b=need.value)

    def call(**kw):
        a = dict(good, **kw)
        r = [byref(a[x]) for x in names]
        return lib.gr_linear_attention_backward(byref(m), *r[:4], a["d"], a["s"], a["si"], a["dso"], *r[4:], a["dsi"],
                                                a["w"], a["b"], NULL)

    assert call() == call(si=NULL, dso=NULL, dsi=NULL) == call(dsi=P(10)) == E("GR_E_DEVICE")
    assert call(dq=rows(0)) == call(dk=rows(4)) == call(dsi=P(9)) == call(dsi=P(1)) == call(dv=rows(10)) == E("GR_E_ALIAS")
    fused = dict(dq=rows(4, 640), dk=rows(4, 640, off=384), dv=rows(4, 640, off=768))
    assert call(**fused) == E("GR_E_DEVICE")
    assert call(**dict(fused, dv=rows(4, 640, off=512))) == E("GR_E_ALIAS")
    assert call(d=NULL) == call(s=NULL) == E("GR_E_NULL")
    assert call(dsi=P(11, 8)) == E("GR_E_ALIGN")


def test_binding_refuses_on_the_host():
    t = torch.zeros(4, 8)
    ids = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: gr.embed(t, ids), lambda: gr.embed_backward(t, ids, 4), lambda: gr.layer_norm(t, t[0]),
                 lambda: gr.linear_attention(t[:, None], t[:, None], t[:, None], t[0])):
        with pytest.raises(ValueError):
            call()


def test_state_gradient_over_the_other_inputs(lib):
    """dstate_in may be dstate_out and nothing else, not at the same address either."""
    m = mixer()
    need = ctypes.c_size_t(0)
    assert lib.gr_linear_attention_workspace_size(byref(m), 1, byref(need)) == 0
    r = [rows(i) for i in range(7)]

    def call(dsi, si=P(9), dso=P(10)):
        return lib.gr_linear_attention_backward(byref(m), *map(byref, r[:4]), P(7), P(8), si, dso, *map(byref, r[4:]),
                                                dsi, P(12), need.value, NULL)

    assert call(P(10)) == call(P(11)) == E("GR_E_DEVICE")
    for k in (7, 8, 9):                     # log_decay, seq_starts, state_in
        assert call(P(k)) == E("GR_E_ALIAS")
    assert call(P(7, -16)) == call(P(8, -16)) == call(P(10, 16)) == E("GR_E_ALIAS")
    assert call(P(9), si=P(9), dso=P(9)) == E("GR_E_ALIAS")


def test_rows_between_other_rows(lib):
    """Outputs between the heads (or tokens) of one fused buffer are taken, in every order of its axes."""
    m = mixer()                              # 20 tokens, 3 heads of 64, bf16
    N, H, d = 20, 3, 64
    need = ctypes.c_size_t(0)
    assert lib.gr_linear_attention_workspace_size(byref(m), 1, byref(need)) == 0

    def prompt(q, k, v, o):
        return lib.gr_linear_attention(byref(m), *map(byref, (q, k, v)), P(4), P(5), NULL, byref(o), NULL, P(8), 1 << 33,
                                       NULL)

    def grads(dq, dk, dv):
        return lib.gr_linear_attention_backward(byref(m), *(byref(rows(i)) for i in range(4)), P(4), P(5), NULL, NULL,
                                                *map(byref, (dq, dk, dv)), NULL, P(8), need.value, NULL)

    for ts, hs, step in ((H * 4 * d, 4 * d, d),                # [N][H][4][d]
                         (H * 4 * d + 64, 4 * d, d),           # the same in a longer row
                         (4 * H * d, d, H * d),                # [N][4][H][d]
                         (4 * d, N * 4 * d, d),                # [H][N][4][d]
                         (d, 4 * N * d, N * d)):               # [H][4][N][d]
        at = [gr.RowsStruct(20 * BIG + 2 * i * step, ts, hs) for i in range(4)]
        for order in ((0, 1, 2, 3), (1, 2, 3, 0), (3, 2, 1, 0)):
            assert prompt(*(at[i] for i in order)) == E("GR_E_DEVICE"), (ts, hs, order)
            assert grads(*(at[i] for i in order[:3])) == E("GR_E_DEVICE"), (ts, hs, order)
        for i in range(3):
            assert prompt(*at[:3], at[i]) == E("GR_E_ALIAS")
            off = gr.RowsStruct(20 * BIG + 2 * i * step + 16, ts, hs)
            assert prompt(*at[:3], off) == E("GR_E_ALIAS"), (ts, hs, i)


def test_rows_that_share_a_byte_are_refused(lib):
    """Small layouts at random against every byte of theirs: what overlaps is never taken."""
    import random
    rng = random.Random(1)
    taken = 0
    for _ in range(4000):
        n, h, d = rng.randint(1, 4), rng.randint(1, 4), 8
        m = mixer(n=n, b=1, h=h, dk=d, dv=d)
        same = rng.random() < 0.7
        strides = [(8 * rng.randint(1, 12), 8 * rng.randint(1, 12)) for _ in range(2)]
        if same:
            strides[1] = strides[0]
        gap = 16 * rng.randint(-40, 40)
        q = gr.RowsStruct(BIG, *strides[0])
        o = gr.RowsStruct(BIG + gap, *strides[1])
        got = lib.gr_linear_attention(byref(m), byref(q), byref(rows(2)), byref(rows(3)), P(4), NULL, NULL, byref(o), NULL,
                                      P(8), 1 << 33, NULL)
        cells = [{base // 16 + (i * ts + j * hs) // 8 for i in range(n) for j in range(h)}
                 for base, (ts, hs) in ((0, strides[0]), (gap, strides[1]))]
        if got == E("GR_E_DEVICE"):
            taken += 1
            assert not cells[0] & cells[1], (n, h, strides, gap)
            assert len(cells[1]) == n * h      # and its own rows do not overlap
        else:
            assert got in (E("GR_E_ALIAS"), E("GR_E_SHAPE"))
    assert taken > 400
