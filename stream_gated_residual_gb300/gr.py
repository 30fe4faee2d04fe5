"""Python binding of libgr_gb300.so: argument marshalling only.

Every step of the Gated Residual read/write runs in the library's CUDA kernels; this module
checks tensor devices, dtypes and contiguity, takes ``data_ptr()`` and the current CUDA stream,
calls the C entry point of the same name and raises ``GRError`` on a non-zero status. PyTorch
supplies device memory and streams. There is no fallback: if the library is missing, every
call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch

from . import build as _build

GR_F32, GR_BF16, GR_FP8 = 0, 1, 2
GR_PARAMS_TAG = 0x47523330304B5031

_DTYPES = {torch.float32: GR_F32, torch.bfloat16: GR_BF16}
# The FP8 branch state is named by torch's e4m3 dtype in shapes and parameter packing; the state
# itself is a pair of uint8 tensors (codes [N,4,D], block exponents [N,4,D/32]).
FP8 = torch.float8_e4m3fn
_SHAPE_DTYPES = {**_DTYPES, FP8: GR_FP8}


class GRError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: status {status} ({status_string(status)})")


class Shape(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int64), ("d_model", ctypes.c_int32),
                ("n_branch", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("state_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class ParamsStruct(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("d_model", ctypes.c_int32),
                ("n_branch", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("state_dtype", ctypes.c_int32), ("tag", ctypes.c_uint64)]


class EmbeddingStruct(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int64), ("n_vocab", ctypes.c_int64),
                ("d_model", ctypes.c_int32), ("n_branch", ctypes.c_int32),
                ("table_dtype", ctypes.c_int32), ("state_dtype", ctypes.c_int32),
                ("id_bits", ctypes.c_int32), ("scale", ctypes.c_float)]


class NormStruct(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int64), ("d_model", ctypes.c_int32),
                ("n_group", ctypes.c_int32), ("dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class MixerStruct(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int64), ("n_seqs", ctypes.c_int32),
                ("n_heads", ctypes.c_int32), ("d_key", ctypes.c_int32),
                ("d_value", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class RowsStruct(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


_LIB = None


def lib_path() -> str:
    return _build.LIB


def load() -> ctypes.CDLL:
    """Load libgr_gb300.so (built by ``__graft_entry__.build()``); raise if it is absent."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(_build.LIB):
        raise RuntimeError(f"{_build.LIB} is missing: build the CUDA library first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    L = ctypes.CDLL(_build.LIB)
    P, S, V = ctypes.POINTER(ParamsStruct), ctypes.POINTER(Shape), ctypes.c_void_p
    sz = ctypes.POINTER(ctypes.c_size_t)
    # the decoder parts take their descriptors as packed bytes (or byref of the structures above)
    E = LN = M = RW = V
    sig = {
        "gr_api_version": ([], ctypes.c_int),
        "gr_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "gr_kernel_path": ([S], ctypes.c_char_p),
        "gr_packed_size": ([S, sz], ctypes.c_int),
        "gr_pack_params": ([S, V, V, V, V, V, ctypes.c_size_t, P, V], ctypes.c_int),
        "gr_read": ([S, V, P, V, V, V], ctypes.c_int),
        "gr_read_ws": ([S, V, P, V, V, V, ctypes.c_size_t, V], ctypes.c_int),
        "gr_step_workspace_size": ([S, sz], ctypes.c_int),
        "gr_write_then_read_ws": ([S, V, V, V, P, V, V, V, ctypes.c_size_t, V], ctypes.c_int),
        "gr_write": ([S, V, V, V, V], ctypes.c_int),
        "gr_write_then_read": ([S, V, V, V, P, V, V, V], ctypes.c_int),
        "gr_read_fixed_gates": ([S, V, V, V, V, V], ctypes.c_int),
        "gr_residual_add_ref": ([ctypes.c_int64, ctypes.c_int32, V, V, V], ctypes.c_int),
        "gr_host_workspace_size": ([S, sz], ctypes.c_int),
        "gr_device_status": ([ctypes.c_int], ctypes.c_int),
        "gr_write_then_read_host": ([S, V, V, V, P, V, V, V, ctypes.c_size_t, V], ctypes.c_int),
        "gr_write_then_read_host_static": ([S, V, V, V, P, V, V, V], ctypes.c_int),
        "gr_selftest_bounded_wait": ([ctypes.c_int64, V], ctypes.c_int),
        "gr_read_backward_workspace_size": ([S, sz], ctypes.c_int),
        "gr_read_backward": ([S] + [V] * 13 + [ctypes.c_size_t, V], ctypes.c_int),
        "gr_write_backward": ([S, V, V, V, V, V, V, V], ctypes.c_int),
        "gr_decompose": ([S, V, V, V, V, V, ctypes.c_int32, V, V, V, V, V, V, V, V],
                         ctypes.c_int),
        "gr_fp8_encode": ([S, V, ctypes.c_int32, V, V, V], ctypes.c_int),
        "gr_fp8_decode": ([S, V, V, V, ctypes.c_int32, V], ctypes.c_int),
        "gr_read_fp8": ([S, V, V, P, V, V, V], ctypes.c_int),
        "gr_write_fp8": ([S, V, V, V, V, V], ctypes.c_int),
        "gr_write_then_read_fp8": ([S, V, V, V, V, P, V, V, V], ctypes.c_int),
        "gr_embed": ([E, V, V, V, V], ctypes.c_int),
        "gr_embed_backward_workspace_size": ([E, sz], ctypes.c_int),
        "gr_embed_backward": ([E, V, V, V, ctypes.c_int, V, ctypes.c_size_t, V], ctypes.c_int),
        "gr_layer_norm": ([LN] + [V] * 7, ctypes.c_int),
        "gr_layer_norm_backward_workspace_size": ([LN, sz], ctypes.c_int),
        "gr_layer_norm_backward": ([LN] + [V] * 9 + [ctypes.c_size_t, V], ctypes.c_int),
        "gr_mixer_path": ([M], ctypes.c_char_p),
        "gr_linear_attention_workspace_size": ([M, ctypes.c_int, sz], ctypes.c_int),
        "gr_linear_attention": ([M, RW, RW, RW, V, V, V, RW, V, V, ctypes.c_size_t, V],
                                ctypes.c_int),
        "gr_linear_attention_step": ([M, RW, RW, RW, V, V, ctypes.c_int64, V, RW, V],
                                     ctypes.c_int),
        "gr_linear_attention_backward": ([M, RW, RW, RW, RW, V, V, V, V, RW, RW, RW, V, V,
                                          ctypes.c_size_t, V], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    _LIB = L
    return L


def status_string(status: int) -> str:
    return load().gr_status_string(int(status)).decode()


def kernel_path(n_tokens: int, d_model: int, rank: int, dtype: torch.dtype) -> str:
    """Which kernel a read or fused step of this shape runs ("fused_bf16",
    "fused_bf16+tiled_bf16", "tiled_bf16", "tc_bf16" (the large-rank path), "tiled_fp8" for
    dtype FP8, or "generic")."""
    return load().gr_kernel_path(ctypes.byref(make_shape(n_tokens, d_model, rank, dtype))).decode()


def _check(status: int, what: str) -> None:
    if status != 0:
        raise GRError(status, what)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t: torch.Tensor | None) -> ctypes.c_void_p:
    return ctypes.c_void_p(None if t is None else t.data_ptr())


def _dev(t: torch.Tensor, name: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _new(stream, shape, dtype: torch.dtype, device) -> torch.Tensor:
    """An output (or a workspace) made here, from the memory of torch's current stream: `stream`,
    where given, is recorded on it, so that the allocator hands the memory out again only after
    the work queued there."""
    t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None:
        t.record_stream(stream)
    return t


def make_shape(n_tokens: int, d_model: int, rank: int, dtype: torch.dtype,
               eps: float = 1e-6) -> Shape:
    if dtype not in _SHAPE_DTYPES:
        raise ValueError(f"state dtype must be float32, bfloat16 or FP8, got {dtype}")
    return Shape(int(n_tokens), int(d_model), 4, int(rank), _SHAPE_DTYPES[dtype], float(eps))


class Params:
    """One GR module's packed parameters: the device buffer and its ``gr_params`` record."""

    def __init__(self, buf: torch.Tensor, st: ParamsStruct, dtype: torch.dtype, eps: float):
        self.buffer = buf
        self.struct = st
        self.dtype = dtype
        self.eps = eps
        self.d_model = st.d_model
        self.rank = st.rank

    def ref(self):
        return ctypes.byref(self.struct)


def packed_size(d_model: int, rank: int, dtype: torch.dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(load().gr_packed_size(ctypes.byref(make_shape(0, d_model, rank, dtype)),
                                 ctypes.byref(n)), "gr_packed_size")
    return n.value


def pack_params(gamma: torch.Tensor, w_down: torch.Tensor, w_up: torch.Tensor,
                w_write: torch.Tensor, dtype: torch.dtype, eps: float = 1e-6,
                stream=None) -> Params:
    """gr_pack_params: fp32 CUDA tensors gamma [4,D], W_d [r,4D], W_u [4D,r], W_w [4,4D]."""
    for t, n in ((gamma, "gamma"), (w_down, "w_down"), (w_up, "w_up"), (w_write, "w_write")):
        _dev(t, n)
        if t.dtype != torch.float32:
            raise ValueError(f"{n} must be float32")
    r, K = w_down.shape
    D = K // 4
    if tuple(gamma.shape) != (4, D) or tuple(w_up.shape) != (K, r) or \
            tuple(w_write.shape) != (4, K):
        raise ValueError("parameter shapes must be gamma [4,D], W_d [r,4D], W_u [4D,r], "
                         "W_w [4,4D]")
    shape = make_shape(0, D, r, dtype, eps)
    nbytes = packed_size(D, r, dtype)
    buf = _new(stream, nbytes + 256, torch.uint8, gamma.device)
    off = (-buf.data_ptr()) % 256
    view = buf[off:off + nbytes]
    st = ParamsStruct()
    _check(load().gr_pack_params(ctypes.byref(shape), _ptr(gamma), _ptr(w_down), _ptr(w_up),
                                 _ptr(w_write), _ptr(view), nbytes, ctypes.byref(st),
                                 _stream(stream)), "gr_pack_params")
    p = Params(view, st, dtype, eps)
    p._keep = buf
    return p


def _state_shape(R: torch.Tensor, params_or_rank, eps: float) -> Shape:
    _dev(R, "R")
    if R.dim() != 3 or R.shape[1] != 4:
        raise ValueError("R must have shape [N, 4, D]")
    rank = params_or_rank.rank if isinstance(params_or_rank, Params) else int(params_or_rank)
    return make_shape(R.shape[0], R.shape[2], rank, R.dtype, eps)


def step_workspace_size(n_tokens: int, d_model: int, rank: int, dtype: torch.dtype) -> int:
    """gr_step_workspace_size: device bytes a read or fused step of this shape needs (0 except on
    the large-rank path)."""
    need = ctypes.c_size_t(0)
    shape = make_shape(n_tokens, d_model, rank, dtype)
    _check(load().gr_step_workspace_size(ctypes.byref(shape), ctypes.byref(need)),
           "gr_step_workspace_size")
    return need.value


def _step_ws(shape: Shape, device, workspace, stream):
    """(pointer, bytes) of the step's workspace: the caller's, else a fresh 256-byte aligned
    buffer when the shape needs one."""
    need = ctypes.c_size_t(0)
    _check(load().gr_step_workspace_size(ctypes.byref(shape), ctypes.byref(need)),
           "gr_step_workspace_size")
    if workspace is not None:
        _dev(workspace, "workspace")
        return _ptr(workspace), workspace.numel() * workspace.element_size(), workspace
    if need.value == 0:
        return ctypes.c_void_p(None), 0, None
    buf = _new(stream, need.value + 256, torch.uint8, device)
    view = buf[(-buf.data_ptr()) % 256:][:need.value]
    return _ptr(view), need.value, buf


def read(R: torch.Tensor, params: Params, x: torch.Tensor | None = None,
         s: torch.Tensor | None = None, stream=None, workspace: torch.Tensor | None = None):
    """gr_read (through gr_read_ws): R [N,4,D] -> (x [N,D], s [N,4] fp32). The large-rank path
    needs a device workspace: the caller's (256-byte aligned), else one allocated here."""
    shape = _state_shape(R, params, params.eps)
    N, _, D = R.shape
    x = _new(stream, (N, D), R.dtype, R.device) if x is None else x
    s = _new(stream, (N, 4), torch.float32, R.device) if s is None else s
    _dev(x, "x")
    _dev(s, "s")
    wp, wn, _keep = _step_ws(shape, R.device, workspace, stream)
    _check(load().gr_read_ws(ctypes.byref(shape), _ptr(R), params.ref(), _ptr(x), _ptr(s), wp,
                             wn, _stream(stream)), "gr_read")
    return x, s


def write(R: torch.Tensor, y: torch.Tensor, s: torch.Tensor, stream=None) -> torch.Tensor:
    """gr_write: R += s_i y in place; returns R."""
    shape = _state_shape(R, 1, 1e-6)
    _dev(y, "y")
    _dev(s, "s")
    _check(load().gr_write(ctypes.byref(shape), _ptr(R), _ptr(y), _ptr(s), _stream(stream)),
           "gr_write")
    return R


def write_then_read(R: torch.Tensor, y: torch.Tensor, s_prev: torch.Tensor, params: Params,
                    x: torch.Tensor | None = None, s_next: torch.Tensor | None = None,
                    stream=None, workspace: torch.Tensor | None = None):
    """gr_write_then_read (through gr_write_then_read_ws): R += s_prev_i y in place, then
    (x, s_next) = read(R, params). Workspace as for read()."""
    shape = _state_shape(R, params, params.eps)
    N, _, D = R.shape
    x = _new(stream, (N, D), R.dtype, R.device) if x is None else x
    s_next = _new(stream, (N, 4), torch.float32, R.device) if s_next is None \
        else s_next
    for t, n in ((y, "y"), (s_prev, "s_prev"), (x, "x"), (s_next, "s_next")):
        _dev(t, n)
    wp, wn, _keep = _step_ws(shape, R.device, workspace, stream)
    _check(load().gr_write_then_read_ws(ctypes.byref(shape), _ptr(R), _ptr(y), _ptr(s_prev),
                                        params.ref(), _ptr(x), _ptr(s_next), wp, wn,
                                        _stream(stream)), "gr_write_then_read")
    return x, s_next


def read_fixed_gates(R: torch.Tensor, gamma: torch.Tensor, G: torch.Tensor, eps: float = 1e-6,
                     x: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gr_read_fixed_gates: x = (1/4) sum_i G_i * RMSNorm(R_i; gamma_i)."""
    shape = _state_shape(R, 1, eps)
    N, _, D = R.shape
    x = _new(stream, (N, D), R.dtype, R.device) if x is None else x
    for t, n in ((gamma, "gamma"), (G, "G"), (x, "x")):
        _dev(t, n)
    _check(load().gr_read_fixed_gates(ctypes.byref(shape), _ptr(R), _ptr(gamma), _ptr(G),
                                      _ptr(x), _stream(stream)), "gr_read_fixed_gates")
    return x


def residual_add_ref(x: torch.Tensor, y: torch.Tensor, stream=None) -> torch.Tensor:
    """gr_residual_add_ref: x += y (single stream), in place."""
    _dev(x, "x")
    _dev(y, "y")
    if x.dtype not in _DTYPES or y.dtype != x.dtype or x.numel() != y.numel():
        raise ValueError("x and y must have the same size and dtype (float32 or bfloat16)")
    _check(load().gr_residual_add_ref(x.numel(), _DTYPES[x.dtype], _ptr(y), _ptr(x),
                                      _stream(stream)), "gr_residual_add_ref")
    return x


def device_status(clear: bool = False) -> int:
    """gr_device_status: 0, or the status code of a bounded device-side wait that ran out."""
    return int(load().gr_device_status(1 if clear else 0))


def selftest_bounded_wait(limit_cycles: int, stream=None) -> None:
    """gr_selftest_bounded_wait: one device-side wait that nothing satisfies gives up after
    limit_cycles and sets the status that device_status() reports."""
    _check(load().gr_selftest_bounded_wait(int(limit_cycles), _stream(stream)),
           "gr_selftest_bounded_wait")


def host_workspace_size(n_tokens: int, d_model: int, dtype: torch.dtype) -> int:
    n = ctypes.c_size_t(0)
    _check(load().gr_host_workspace_size(ctypes.byref(make_shape(n_tokens, d_model, 1, dtype)),
                                         ctypes.byref(n)), "gr_host_workspace_size")
    return n.value


def write_then_read_host(R: torch.Tensor, y: torch.Tensor, s_prev: torch.Tensor,
                         params: Params, x: torch.Tensor, s_next: torch.Tensor,
                         workspace: torch.Tensor, stream=None):
    """gr_write_then_read_host on CPU tensors (pinned for asynchronous copies); `workspace` is
    a CUDA uint8 tensor of at least host_workspace_size() bytes, 256-byte aligned."""
    for t, n in ((R, "R"), (y, "y"), (s_prev, "s_prev"), (x, "x"), (s_next, "s_next")):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous CPU tensor")
    N, _, D = R.shape
    shape = make_shape(N, D, params.rank, R.dtype, params.eps)
    _check(load().gr_write_then_read_host(
        ctypes.byref(shape), _ptr(R), _ptr(y), _ptr(s_prev), params.ref(), _ptr(x), _ptr(s_next),
        _ptr(workspace), workspace.numel(), _stream(stream)), "gr_write_then_read_host")
    return x, s_next


def write_then_read_host_static(R: torch.Tensor, y: torch.Tensor, s_prev: torch.Tensor,
                                params: Params, x: torch.Tensor, s_next: torch.Tensor,
                                stream=None):
    """gr_write_then_read_host_static on CPU tensors (pinned for asynchronous copies), staged
    through the library's fixed 32 MiB device workspace (GR_STATIC_WORKSPACE_BYTES), for callers
    that cannot allocate device memory: a host program without a device allocator, a process
    whose device memory a pool already holds, or a decode loop that cannot afford the device-wide
    synchronisation of cudaFree. Nothing is allocated; shapes that need more than the workspace
    raise GR_E_SIZE, and calls must not overlap in time (they share the workspace)."""
    for t, n in ((R, "R"), (y, "y"), (s_prev, "s_prev"), (x, "x"), (s_next, "s_next")):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous CPU tensor")
    N, _, D = R.shape
    shape = make_shape(N, D, params.rank, R.dtype, params.eps)
    _check(load().gr_write_then_read_host_static(
        ctypes.byref(shape), _ptr(R), _ptr(y), _ptr(s_prev), params.ref(), _ptr(x), _ptr(s_next),
        _stream(stream)), "gr_write_then_read_host_static")
    return x, s_next


# ---- backward (training) ------------------------------------------------------------------------

def read_backward(R: torch.Tensor, gamma: torch.Tensor, w_down: torch.Tensor, w_up: torch.Tensor,
                  w_write: torch.Tensor, dx: torch.Tensor, ds: torch.Tensor, eps: float = 1e-6,
                  workspace: torch.Tensor | None = None, stream=None):
    """gr_read_backward: dL/dR [N,4,D] fp32 and the parameter gradients (dict like the
    parameters: gamma, w_down, w_up, w_write; fp32) given dL/dx [N,D] and dL/ds [N,4] (fp32).
    The parameters are the fp32 tensors (not the packed buffer)."""
    _dev(R, "R")
    N, _, D = R.shape
    r = w_down.shape[0]
    shape = make_shape(N, D, r, R.dtype, eps)
    for t, n in ((gamma, "gamma"), (w_down, "w_down"), (w_up, "w_up"), (w_write, "w_write"),
                 (dx, "dx"), (ds, "ds")):
        _dev(t, n)
        if t.dtype != torch.float32:
            raise ValueError(f"{n} must be float32")
    need = ctypes.c_size_t(0)
    _check(load().gr_read_backward_workspace_size(ctypes.byref(shape), ctypes.byref(need)),
           "gr_read_backward_workspace_size")
    if workspace is None:
        buf = _new(stream, need.value + 256, torch.uint8, R.device)
        workspace = buf[(-buf.data_ptr()) % 256:][:need.value]
    dev = R.device
    dR = _new(stream, (N, 4, D), torch.float32, dev)
    g = {k: _new(stream, t.shape, torch.float32, dev)
         for k, t in (("gamma", gamma), ("w_down", w_down), ("w_up", w_up), ("w_write", w_write))}
    _check(load().gr_read_backward(
        ctypes.byref(shape), _ptr(R), _ptr(gamma), _ptr(w_down), _ptr(w_up), _ptr(w_write),
        _ptr(dx), _ptr(ds), _ptr(dR), _ptr(g["gamma"]), _ptr(g["w_down"]), _ptr(g["w_up"]),
        _ptr(g["w_write"]), _ptr(workspace), workspace.numel(), _stream(stream)),
        "gr_read_backward")
    return dR, g


def write_backward(dR_next: torch.Tensor, y: torch.Tensor, s: torch.Tensor, stream=None):
    """gr_write_backward: (dR, dy, ds) from dL/dR' [N,4,D] fp32, y [N,D] (state dtype), s [N,4]."""
    for t, n in ((dR_next, "dR_next"), (y, "y"), (s, "s")):
        _dev(t, n)
    N, _, D = dR_next.shape
    shape = make_shape(N, D, 1, y.dtype)
    dR = _new(stream, dR_next.shape, dR_next.dtype, dR_next.device)
    dy = _new(stream, (N, D), torch.float32, dR_next.device)
    ds = _new(stream, (N, 4), torch.float32, dR_next.device)
    _check(load().gr_write_backward(ctypes.byref(shape), _ptr(dR_next), _ptr(y), _ptr(s),
                                    _ptr(dR), _ptr(dy), _ptr(ds), _stream(stream)),
           "gr_write_backward")
    return dR, dy, ds


# ---- contribution decomposition ---------------------------------------------------------------

def decompose(R: torch.Tensor, gamma: torch.Tensor, w_down: torch.Tensor, w_up: torch.Tensor,
              w_write: torch.Tensor, y: torch.Tensor | None, s: torch.Tensor | None,
              R0: torch.Tensor | None = None, eps: float = 1e-6, branch_norm: bool = True,
              pi: bool = True, stream=None) -> dict:
    """gr_decompose at one reader: R [N,4,D] the state it reads, its fp32 parameters, the
    writers' outputs y [U,N,D] (state dtype) and write strengths s [U,N,4] (fp32), optionally
    the initial state R0 [N,4,D]. Returns fp32 tensors: norm [N,U], branch_norm [N,U,4] and pi
    [N,U] (when asked), a0_norm [N] (with R0)."""
    _dev(R, "R")
    N, _, D = R.shape
    r = w_down.shape[0]
    shape = make_shape(N, D, r, R.dtype, eps)
    for t, n in ((gamma, "gamma"), (w_down, "w_down"), (w_up, "w_up"), (w_write, "w_write")):
        _dev(t, n)
        if t.dtype != torch.float32:
            raise ValueError(f"{n} must be float32")
    U = 0 if y is None else y.shape[0]
    if U:
        _dev(y, "y")
        _dev(s, "s")
        if y.dtype != R.dtype or tuple(y.shape) != (U, N, D) or tuple(s.shape) != (U, N, 4) \
                or s.dtype != torch.float32:
            raise ValueError("y must be [U, N, D] in the state dtype and s [U, N, 4] float32")
    if R0 is not None:
        _dev(R0, "R0")
        if R0.dtype != R.dtype or R0.shape != R.shape:
            raise ValueError("R0 must match R")
    dev = R.device
    out = {"norm": _new(stream, (N, U), torch.float32, dev)}
    if branch_norm:
        out["branch_norm"] = _new(stream, (N, U, 4), torch.float32, dev)
    if pi:
        out["pi"] = _new(stream, (N, U), torch.float32, dev)
    if R0 is not None:
        out["a0_norm"] = _new(stream, (N,), torch.float32, dev)

    def p(k):
        t = out.get(k)
        return _ptr(t) if t is not None and t.numel() else None

    _check(load().gr_decompose(
        ctypes.byref(shape), _ptr(R), _ptr(gamma), _ptr(w_down), _ptr(w_up), _ptr(w_write), U,
        _ptr(y) if U else None, _ptr(s) if U else None, _ptr(R0) if R0 is not None else None,
        p("norm"), p("branch_norm"), p("pi"), p("a0_norm"), _stream(stream)), "gr_decompose")
    return out


# ---- FP8 branch state (e4m3 codes, one power-of-two exponent per 32-channel block) ------------

def _fp8_state(codes: torch.Tensor, scales: torch.Tensor):
    _dev(codes, "codes")
    _dev(scales, "scales")
    if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise ValueError("codes and scales must be uint8")
    if codes.dim() != 3 or codes.shape[1] != 4 or codes.shape[2] % 32:
        raise ValueError("codes must have shape [N, 4, D] with D a multiple of 32")
    N, _, D = codes.shape
    if tuple(scales.shape) != (N, 4, D // 32):
        raise ValueError("scales must have shape [N, 4, D/32]")
    return N, D


def fp8_encode(R: torch.Tensor, codes: torch.Tensor | None = None,
               scales: torch.Tensor | None = None, stream=None):
    """gr_fp8_encode: a bf16 or fp32 state R [N,4,D] -> (codes [N,4,D], scales [N,4,D/32])."""
    _dev(R, "R")
    if R.dtype not in _DTYPES or R.dim() != 3 or R.shape[1] != 4:
        raise ValueError("R must be a float32 or bfloat16 tensor of shape [N, 4, D]")
    N, _, D = R.shape
    codes = _new(stream, (N, 4, D), torch.uint8, R.device) if codes is None else codes
    scales = _new(stream, (N, 4, D // 32), torch.uint8, R.device) if scales is None \
        else scales
    _fp8_state(codes, scales)
    shape = make_shape(N, D, 1, FP8)
    _check(load().gr_fp8_encode(ctypes.byref(shape), _ptr(R), _DTYPES[R.dtype], _ptr(codes),
                                _ptr(scales), _stream(stream)), "gr_fp8_encode")
    return codes, scales


def fp8_decode(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.float32,
               out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gr_fp8_decode: (codes, scales) -> the state's values [N,4,D] in float32 or bfloat16."""
    N, D = _fp8_state(codes, scales)
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    out = _new(stream, (N, 4, D), dtype, codes.device) if out is None else out
    _dev(out, "out")
    shape = make_shape(N, D, 1, FP8)
    _check(load().gr_fp8_decode(ctypes.byref(shape), _ptr(codes), _ptr(scales), _ptr(out),
                                _DTYPES[dtype], _stream(stream)), "gr_fp8_decode")
    return out


def read_fp8(codes: torch.Tensor, scales: torch.Tensor, params: Params,
             x: torch.Tensor | None = None, s: torch.Tensor | None = None, stream=None):
    """gr_read_fp8: FP8 state -> (x [N,D] bf16, s [N,4] fp32)."""
    N, D = _fp8_state(codes, scales)
    shape = make_shape(N, D, params.rank, FP8, params.eps)
    x = _new(stream, (N, D), torch.bfloat16, codes.device) if x is None else x
    s = _new(stream, (N, 4), torch.float32, codes.device) if s is None else s
    _dev(x, "x")
    _dev(s, "s")
    _check(load().gr_read_fp8(ctypes.byref(shape), _ptr(codes), _ptr(scales), params.ref(),
                              _ptr(x), _ptr(s), _stream(stream)), "gr_read_fp8")
    return x, s


def write_fp8(codes: torch.Tensor, scales: torch.Tensor, y: torch.Tensor, s: torch.Tensor,
              stream=None):
    """gr_write_fp8: R += s_i y on the FP8 state (y bf16 [N,D]), in place."""
    N, D = _fp8_state(codes, scales)
    _dev(y, "y")
    _dev(s, "s")
    shape = make_shape(N, D, 1, FP8)
    _check(load().gr_write_fp8(ctypes.byref(shape), _ptr(codes), _ptr(scales), _ptr(y), _ptr(s),
                               _stream(stream)), "gr_write_fp8")
    return codes, scales


def write_then_read_fp8(codes: torch.Tensor, scales: torch.Tensor, y: torch.Tensor,
                        s_prev: torch.Tensor, params: Params, x: torch.Tensor | None = None,
                        s_next: torch.Tensor | None = None, stream=None):
    """gr_write_then_read_fp8: the write in place on the FP8 state, then the read with
    `params` -> (x [N,D] bf16, s_next [N,4] fp32)."""
    N, D = _fp8_state(codes, scales)
    shape = make_shape(N, D, params.rank, FP8, params.eps)
    x = _new(stream, (N, D), torch.bfloat16, codes.device) if x is None else x
    s_next = _new(stream, (N, 4), torch.float32, codes.device) if s_next is None \
        else s_next
    for t, n in ((y, "y"), (s_prev, "s_prev"), (x, "x"), (s_next, "s_next")):
        _dev(t, n)
    _check(load().gr_write_then_read_fp8(ctypes.byref(shape), _ptr(codes), _ptr(scales), _ptr(y),
                                         _ptr(s_prev), params.ref(), _ptr(x), _ptr(s_next),
                                         _stream(stream)), "gr_write_then_read_fp8")
    return x, s_next


# ---- the parts of a decoder around the Gated Residual: embedding, layer norm, linear attention ----
#
# These calls are also made for a few tokens at a time, where the binding itself is what a call costs.
# Descriptors are packed bytes, kept by their values (numbers of Python: a tensor would be kept by its
# identity); workspace sizes are kept by the descriptor (both are pure functions of the arguments), and
# pointers go as plain integers.

_EMBED = struct.Struct("=qqiiiiif")    # gr_embedding
_NORM = struct.Struct("=qiiif")        # gr_norm
_MIXER = struct.Struct("=qiiiiif")     # gr_mixer
_ROWS = struct.Struct("=Qqq")          # gr_rows
_embed_desc = functools.lru_cache(1024)(_EMBED.pack)
_norm_desc = functools.lru_cache(1024)(_NORM.pack)
_mixer_desc = functools.lru_cache(1024)(_MIXER.pack)


_current_device = torch._C._cuda_getDevice


@functools.cache
def _several_devices() -> bool:
    return torch.cuda.device_count() > 1


def _raw_stream(stream, t: torch.Tensor, *others: torch.Tensor | None) -> int:
    """cudaStream_t of `stream`, or of torch's current stream. The library launches on the current
    device, so all tensors of the call have to be there (asked where the process sees several)."""
    device = t.get_device()
    if _several_devices():
        if device != _current_device():
            raise ValueError(f"the tensors are on device {device}, the current device is "
                             f"{_current_device()}")
        for o in others:
            if o is not None and o.get_device() != device:
                raise ValueError("all tensors of a call must be on one device, got devices "
                                 f"{device} and {o.get_device()}")
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device)


def _call(name: str, *args) -> None:
    status = getattr(_LIB or load(), name)(*args)
    if status != 0:
        raise GRError(status, name)


@functools.lru_cache(1024)
def _need(name: str, desc: bytes, *args) -> int:
    """Bytes of a workspace-size entry (a function of the descriptor alone)."""
    n = ctypes.c_size_t(0)
    _call(name, desc, *args, ctypes.byref(n))
    return n.value


def _ws(need: int, workspace: torch.Tensor | None, like: torch.Tensor, stream):
    """(pointer, bytes, tensor) of the call's workspace: the caller's, else a fresh one (torch's
    allocations start at multiples of 512 bytes) that `stream` is recorded on."""
    if workspace is not None:
        _dev(workspace, "workspace")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    if need == 0:
        return None, 0, None
    buf = _new(stream, need, torch.uint8, like.device)
    return buf.data_ptr(), need, buf


def _opt(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _f32(t: torch.Tensor | None, name: str, shape=None) -> None:
    if t is None:
        return
    if not t.is_cuda or not t.is_contiguous():
        _dev(t, name)
    if t.dtype != torch.float32:
        raise ValueError(f"{name} must be float32")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")


def _ids(ids: torch.Tensor) -> int:
    _dev(ids, "ids")
    if ids.dtype == torch.int64:
        return 64
    if ids.dtype != torch.int32:
        raise ValueError("ids must be int32 or int64")
    return 32


def embed(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, branches: int = 4,
          dtype: torch.dtype | None = None, out: torch.Tensor | None = None, stream=None):
    """gr_embed: the state a stack starts from, R[t, i] = scale * table[ids[t]] in every branch:
    [N, 4, D], or [N, D] with branches=1; N = ids.numel(), dtype the table's unless given. An id
    outside the table gives a zero row."""
    _dev(table, "table")
    dtype = table.dtype if dtype is None else dtype
    if table.dtype not in _DTYPES or dtype not in _DTYPES or table.dim() != 2:
        raise ValueError("table must be a float32 or bfloat16 tensor [V, D] and dtype one of these")
    bits = _ids(ids)
    (V, D), N = table.shape, ids.numel()
    shape = (N, D) if branches == 1 else (N, branches, D)
    if out is None:
        out = _new(stream, shape, dtype, table.device)
    else:
        _dev(out, "out")
        if out.shape != shape or out.dtype != dtype:
            raise ValueError(f"out must be {dtype} of shape {list(shape)}")
    e = _embed_desc(N, V, D, int(branches), _DTYPES[table.dtype], _DTYPES[dtype], bits, float(scale))
    _call("gr_embed", e, table.data_ptr(), ids.data_ptr(), out.data_ptr(),
          _raw_stream(stream, table, ids, out))
    return out


def embed_backward(dR: torch.Tensor, ids: torch.Tensor, n_vocab: int, scale: float = 1.0,
                   dtable: torch.Tensor | None = None, accumulate: bool = False,
                   workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gr_embed_backward: the table's gradient [n_vocab, D] fp32 from dR [N, 4, D] or [N, D] fp32;
    rows of equal ids are summed in a fixed order. accumulate=True adds to the given dtable."""
    _f32(dR, "dR")
    bits = _ids(ids)
    nd = dR.dim()
    if nd not in (2, 3) or dR.shape[0] != ids.numel():
        raise ValueError("dR must be [N, 4, D] or [N, D] with N = ids.numel()")
    if accumulate and dtable is None:
        raise ValueError("accumulate needs the dtable to add to")
    N, D = dR.shape[0], dR.shape[-1]
    if dtable is None:
        dtable = _new(stream, (n_vocab, D), torch.float32, dR.device)
    else:
        _f32(dtable, "dtable", (n_vocab, D))
    e = _embed_desc(N, int(n_vocab), D, 1 if nd == 2 else dR.shape[1], GR_F32, GR_F32, bits,
                    float(scale))
    wp, wn, _keep = _ws(_need("gr_embed_backward_workspace_size", e), workspace, dR, stream)
    _call("gr_embed_backward", e, dR.data_ptr(), ids.data_ptr(), dtable.data_ptr(),
          1 if accumulate else 0, wp, wn, _raw_stream(stream, dR, ids, dtable, workspace))
    return dtable


def _norm_rows(x: torch.Tensor, weight: torch.Tensor, eps: float) -> bytes:
    if not x.is_cuda or not x.is_contiguous():
        _dev(x, "x")
    if x.dtype not in _DTYPES or x.dim() not in (2, 3):
        raise ValueError("x must be a float32 or bfloat16 tensor [N, D] or [N, 4, D]")
    shape = x.shape
    _f32(weight, "weight", shape[1:])
    return _norm_desc(shape[0], shape[-1], 1 if len(shape) == 2 else shape[1], _DTYPES[x.dtype],
                      float(eps))


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
               eps: float = 1e-5, y: torch.Tensor | None = None, stats: bool = False, stream=None):
    """gr_layer_norm over the last axis of x [N, D] (weight, bias [D]) or of every branch of
    x [N, 4, D] (weight, bias [4, D]); weight and bias fp32. Returns y, or (y, mean, rstd) with
    stats=True (fp32, what the gradient needs). y may be x."""
    n = _norm_rows(x, weight, eps)
    _f32(bias, "bias", x.shape[1:])
    if y is None:
        y = _new(stream, x.shape, x.dtype, x.device)
    else:
        _dev(y, "y")
        if y.shape != x.shape or y.dtype != x.dtype:
            raise ValueError("y must match x")
    mean = rstd = None
    if stats:
        mean = _new(stream, x.shape[:-1], torch.float32, x.device)
        rstd = _new(stream, x.shape[:-1], torch.float32, x.device)
    _call("gr_layer_norm", n, x.data_ptr(), weight.data_ptr(), _opt(bias), y.data_ptr(), _opt(mean),
          _opt(rstd), _raw_stream(stream, x, weight, bias, y))
    return (y, mean, rstd) if stats else y


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                        mean: torch.Tensor, rstd: torch.Tensor, bias: bool = True,
                        dx: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        stream=None):
    """gr_layer_norm_backward: (dx like x but fp32, dweight, dbias or None) from dy (fp32, x's shape)
    and the forward's mean and rstd. dx may be dy."""
    n = _norm_rows(x, weight, 0.0)
    shape = x.shape
    _f32(dy, "dy", shape)
    _f32(mean, "mean", shape[:-1])
    _f32(rstd, "rstd", shape[:-1])
    if dx is None:
        dx = _new(stream, shape, torch.float32, x.device)
    else:
        _f32(dx, "dx", shape)
    dweight = _new(stream, shape[1:], torch.float32, x.device)
    dbias = _new(stream, shape[1:], torch.float32, x.device) if bias else None
    wp, wn, _keep = _ws(_need("gr_layer_norm_backward_workspace_size", n), workspace, x, stream)
    _call("gr_layer_norm_backward", n, dy.data_ptr(), x.data_ptr(), weight.data_ptr(),
          mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), dweight.data_ptr(), _opt(dbias), wp, wn,
          _raw_stream(stream, x, dy, weight, mean, rstd, dx, workspace))
    return dx, dweight, dbias


def _rows(t: torch.Tensor, name: str, N: int, H: int, d: int, dtype: torch.dtype) -> bytes:
    """gr_rows of a [N, H, d] tensor with contiguous channels at any token and head stride."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.shape != (N, H, d) or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} of shape {[N, H, d]}, got {t.dtype} of "
                         f"{list(t.shape)}")
    ts, hs, cs = t.stride()
    if cs != 1 and t.numel():
        raise ValueError(f"the channels of {name} must be contiguous")
    return _ROWS.pack(t.data_ptr(), ts, hs)


def _mixer(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
           scale: float | None, n_seqs: int):
    """(N, H, dk, dv, descriptor, rows of q, k and v) of a linear-attention call."""
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, v must have shape [N, H, d]")
    (N, H, dk), dv, dtype = q.shape, v.shape[2], q.dtype
    if dtype not in _DTYPES:
        raise ValueError("q, k, v must be float32 or bfloat16")
    rows = (_rows(q, "q", N, H, dk, dtype), _rows(k, "k", N, H, dk, dtype),
            _rows(v, "v", N, H, dv, dtype))
    _f32(log_decay, "log_decay", (H,))
    m = _mixer_desc(N, n_seqs, H, dk, dv, _DTYPES[dtype],
                    dk ** -0.5 if scale is None else float(scale))
    return N, H, dk, dv, m, rows


def _seqs(seq_starts: torch.Tensor | None) -> int:
    if seq_starts is None:
        return 1
    _dev(seq_starts, "seq_starts")
    if seq_starts.dtype != torch.int32 or seq_starts.dim() != 1 or seq_starts.numel() < 1:
        raise ValueError("seq_starts must be int32 [n_seqs + 1]")
    return seq_starts.numel() - 1


def mixer_path(n_tokens: int, n_heads: int, d_key: int, d_value: int, dtype: torch.dtype) -> str:
    """Which kernels a linear-attention prompt of this shape runs: "mixer_tc" or "mixer_simt"."""
    m = _mixer_desc(int(n_tokens), 1, int(n_heads), int(d_key), int(d_value), _DTYPES.get(dtype, -1),
                    1.0)
    return load().gr_mixer_path(m).decode()


def linear_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                     scale: float | None = None, seq_starts: torch.Tensor | None = None,
                     state: torch.Tensor | None = None, o: torch.Tensor | None = None,
                     state_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None):
    """gr_linear_attention: q, k [N, H, dk], v [N, H, dv] (strided views allowed) of the packed
    sequences seq_starts (int32 [B + 1]; None: one sequence), log_decay [H] fp32 <= 0, scale
    dk ** -0.5 unless given, state [B, H, dk, dv] fp32 before each sequence or None. Returns
    (o [N, H, dv], state_out [B, H, dk, dv] fp32 after each sequence). state_out may be state."""
    B = _seqs(seq_starts)
    N, H, dk, dv, m, rows = _mixer(q, k, v, log_decay, scale, B)
    _f32(state, "state", (B, H, dk, dv))
    if o is None:
        o = _new(stream, (N, H, dv), q.dtype, q.device)
    if state_out is None:
        state_out = _new(stream, (B, H, dk, dv), torch.float32, q.device)
    else:
        _f32(state_out, "state_out", (B, H, dk, dv))
    orow = _rows(o, "o", N, H, dv, q.dtype)
    wp, wn, _keep = _ws(_need("gr_linear_attention_workspace_size", m, 0), workspace, q, stream)
    _call("gr_linear_attention", m, *rows, log_decay.data_ptr(), _opt(seq_starts), _opt(state), orow,
          state_out.data_ptr(), wp, wn,
          _raw_stream(stream, q, k, v, log_decay, seq_starts, state, o, state_out, workspace))
    return o, state_out


def linear_attention_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                          log_decay: torch.Tensor, state: torch.Tensor,
                          scale: float | None = None, slots: torch.Tensor | None = None,
                          o: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gr_linear_attention_step: one token of each of N requests. state [slots, H, dk, dv] fp32 is
    updated in place; request n uses state[slots[n]] (int32; None: state[n]). Returns o [N, H, dv];
    a slot outside the states leaves them alone and gives o = 0."""
    N, H, dk, dv, m, rows = _mixer(q, k, v, log_decay, scale, 0)
    if state.dim() != 4 or state.shape[1:] != (H, dk, dv):
        raise ValueError(f"state must be [slots, {H}, {dk}, {dv}]")
    _f32(state, "state")
    if slots is not None:
        _dev(slots, "slots")
        if slots.dtype != torch.int32 or slots.shape != (N,):
            raise ValueError("slots must be int32 [N]")
    elif state.shape[0] < N:
        raise ValueError("state must hold a slot for every request")
    if o is None:
        o = _new(stream, (N, H, dv), q.dtype, q.device)
    _call("gr_linear_attention_step", m, *rows, log_decay.data_ptr(), state.data_ptr(),
          state.shape[0], _opt(slots), _rows(o, "o", N, H, dv, q.dtype),
          _raw_stream(stream, q, k, v, log_decay, state, slots, o))
    return o


def linear_attention_backward(do: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                              log_decay: torch.Tensor, scale: float | None = None,
                              seq_starts: torch.Tensor | None = None,
                              state: torch.Tensor | None = None,
                              dstate: torch.Tensor | None = None, out=None,
                              workspace: torch.Tensor | None = None, stream=None,
                              dstate_in: torch.Tensor | None = None):
    """gr_linear_attention_backward: (dq, dk, dv, dstate_in) from do [N, H, dv] and, optionally, the
    gradient dstate [B, H, dk, dv] of state_out. dq, dk, dv come in q's dtype (out: a triple to write,
    strided views allowed); dstate_in, the gradient of state, is made where dstate or state is given, or
    written to the tensor given for it, which may be dstate."""
    B = _seqs(seq_starts)
    N, H, dk, dv, m, rows = _mixer(q, k, v, log_decay, scale, B)
    _f32(state, "state", (B, H, dk, dv))
    _f32(dstate, "dstate", (B, H, dk, dv))
    dorow = _rows(do, "do", N, H, dv, q.dtype)
    if out is None:
        out = [_new(stream, (N, H, d), q.dtype, q.device) for d in (dk, dk, dv)]
    outs = [_rows(t, n, N, H, d, q.dtype)
            for t, n, d in zip(out, ("dq", "dk", "dv"), (dk, dk, dv))]
    if dstate_in is not None:
        _f32(dstate_in, "dstate_in", (B, H, dk, dv))
    elif state is not None or dstate is not None:
        dstate_in = _new(stream, (B, H, dk, dv), torch.float32, q.device)
    wp, wn, _keep = _ws(_need("gr_linear_attention_workspace_size", m, 1), workspace, q, stream)
    _call("gr_linear_attention_backward", m, dorow, *rows, log_decay.data_ptr(), _opt(seq_starts),
          _opt(state), _opt(dstate), *outs, _opt(dstate_in), wp, wn,
          _raw_stream(stream, q, do, k, v, log_decay, seq_starts, state, dstate, *out, dstate_in,
                      workspace))
    return (*out, dstate_in)
