"""Thin Python binding of the C ABI in include/moe.h (libmoe.so).

Argument marshalling only: every function here checks tensor devices, dtypes
and shapes, allocates missing outputs with torch, and calls the C entry point of
the same name on the current CUDA stream.  Every step of the layer runs in the
library's CUDA kernels; there is no fallback path.  If libmoe.so is missing the
first call raises ImportError.

Shapes follow the C header: `shape = (T, d, d_ff, E, k)`.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_CUDA = 4
MOE_ERR_DEVICE_TIMEOUT = 5

# Entry points declared in include/moe.h.
EXPORTS = (
    "moe_status_string", "moe_check_shape", "moe_expert_workspace_bytes",
    "moe_forward_workspace_bytes", "moe_forward_kernel_count", "moe_forward_hostio_workspace_bytes",
    "moe_route",
    "moe_dispatch", "moe_expert_swiglu", "moe_expert_swiglu_bias", "moe_expert_swiglu_stall_test",
    "moe_combine", "moe_forward", "moe_forward_bias", "moe_forward_profiled", "moe_forward_hostio", "moe_forward_hostio_stall_test",
    "moe_forward_hostio_batches_workspace_bytes", "moe_forward_hostio_batches",
    "moe_forward_hostio_batches_stall_test",
    "moe_forward_static",
    "moe_aux_loss", "moe_block_workspace_bytes", "moe_block_forward", "moe_read_device_status",
    "moe_check_scoring", "moe_route_scored", "moe_route_scored_backward", "moe_check_shape_int8",
    "moe_quantize_weights_int8", "moe_dispatch_int8", "moe_expert_swiglu_int8_workspace_bytes",
    "moe_expert_swiglu_int8", "moe_expert_swiglu_int8_stall_test", "moe_combine_bf16",
    "moe_forward_int8_workspace_bytes", "moe_forward_int8",
)

MOE_STATIC_SCRATCH_BYTES = 8 << 20


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32)]


class MoeScoring(ctypes.Structure):
    """Scores, groups and gates of moe_route_scored (moe_scoring of include/moe.h).

    score: "softmax" over the row's logits or their "sigmoid"s; n_group groups of E / n_group
    consecutive experts, of which the topk_group best stay, a group's value being
    its largest choice (group_top = 1) or the sum of its two largest (2); renorm
    divides a token's gates by their sum; scale multiplies them."""
    _fields_ = [("score", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("scale", ctypes.c_float)]
    SCORES = {"softmax": 0, "sigmoid": 1}

    def __init__(self, score="softmax", n_group=1, topk_group=1, group_top=1, renorm=True,
                 scale=1.0):
        if score not in self.SCORES:
            raise ValueError(f"score must be one of {tuple(self.SCORES)}, got {score!r}")
        super().__init__(self.SCORES[score], int(n_group), int(topk_group), int(group_top),
                         int(bool(renorm)), float(scale))


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)}")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libmoe.so (raises ImportError when it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m sparse_mixture_experts_05_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        I = ctypes.c_int
        S = MoeShape
        Z = ctypes.c_size_t
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_status_string.argtypes = [I]
        L.moe_check_shape.restype = I
        L.moe_check_shape.argtypes = [S]
        for fn in ("moe_expert_workspace_bytes", "moe_forward_workspace_bytes",
                   "moe_forward_hostio_workspace_bytes", "moe_block_workspace_bytes",
                   "moe_forward_hostio_batches_workspace_bytes"):
            getattr(L, fn).restype = Z
            getattr(L, fn).argtypes = [S]
        L.moe_forward_kernel_count.restype = I
        L.moe_forward_kernel_count.argtypes = [S]
        L.moe_route.restype = I
        L.moe_route.argtypes = [S, P, P, P, P, P, P, P]
        L.moe_dispatch.restype = I
        L.moe_dispatch.argtypes = [S, P, P, P, P, P, P, P]
        L.moe_expert_swiglu.restype = I
        L.moe_expert_swiglu.argtypes = [S, P, P, P, P, P, P, P, P, Z, P]
        L.moe_expert_swiglu_stall_test.restype = I
        L.moe_expert_swiglu_stall_test.argtypes = [S, P, P, P, P, P, P, P, P, Z, I,
                                                   ctypes.c_uint64, P]
        L.moe_combine.restype = I
        L.moe_expert_swiglu_bias.restype = I
        L.moe_expert_swiglu_bias.argtypes = [S, P, P, P, P, P, P, P, P, P, P, P, Z, P]
        L.moe_forward_bias.restype = I
        L.moe_forward_bias.argtypes = [S, P, P, P, P, P, P, P, P, P, P, P, P, P, Z, P]
        L.moe_combine.argtypes = [S, P, P, P, P, P]
        L.moe_forward.restype = I
        L.moe_forward.argtypes = [S, P, P, P, P, P, P, P, P, P, P, Z, P]
        L.moe_forward_profiled.restype = I
        L.moe_forward_profiled.argtypes = [S, P, P, P, P, P, P, P, P, Z, P, I, P]
        L.moe_forward_hostio.restype = I
        L.moe_forward_hostio.argtypes = [S, P, P, P, P, P, P, P, P, Z, P]
        L.moe_forward_hostio_batches.restype = I
        L.moe_forward_hostio_batches.argtypes = [S, I, P, P, P, P, P, P, P, P, Z, P]
        L.moe_forward_hostio_batches_stall_test.restype = I
        L.moe_forward_hostio_batches_stall_test.argtypes = [S, I, P, P, P, P, P, P, P, P, Z, I,
                                                            I, ctypes.c_uint64, P]
        L.moe_forward_hostio_stall_test.restype = I
        L.moe_forward_hostio_stall_test.argtypes = [S, P, P, P, P, P, P, P, P, Z, I, I,
                                                    ctypes.c_uint64, P]
        L.moe_forward_static.restype = I
        L.moe_forward_static.argtypes = [S, P, P, P, P, P, P, P, P, P]
        L.moe_block_forward.restype = I
        L.moe_block_forward.argtypes = [S, P, P, ctypes.c_float, P, P, P, P, P, P, P, Z, P]
        L.moe_aux_loss.restype = I
        L.moe_aux_loss.argtypes = [S, P, P, P, P, P, P, P]
        C = MoeScoring
        L.moe_check_scoring.restype = I
        L.moe_check_scoring.argtypes = [S, C]
        L.moe_check_shape_int8.restype = I
        L.moe_check_shape_int8.argtypes = [S]
        for fn in ("moe_expert_swiglu_int8_workspace_bytes", "moe_forward_int8_workspace_bytes"):
            getattr(L, fn).restype = Z
            getattr(L, fn).argtypes = [S]
        L.moe_route_scored.restype = I
        L.moe_route_scored.argtypes = [S, C, P, I, P, P, P, P, P]
        L.moe_route_scored_backward.restype = I
        L.moe_route_scored_backward.argtypes = [S, C, P, I, P, P, P, P]
        L.moe_quantize_weights_int8.restype = I
        L.moe_quantize_weights_int8.argtypes = [I, I, I, P, P, P, P]
        L.moe_dispatch_int8.restype = I
        L.moe_dispatch_int8.argtypes = [S, P, P, P, P, P, P, P, P]
        L.moe_expert_swiglu_int8.restype = I
        L.moe_expert_swiglu_int8.argtypes = [S] + [P] * 11 + [Z, P]
        L.moe_expert_swiglu_int8_stall_test.restype = I
        L.moe_expert_swiglu_int8_stall_test.argtypes = [S] + [P] * 11 + [Z, I, ctypes.c_uint64, P]
        L.moe_combine_bf16.restype = I
        L.moe_combine_bf16.argtypes = [S, P, P, P, P, P]
        L.moe_forward_int8.restype = I
        L.moe_forward_int8.argtypes = [S, P, P, I, C, P, P] + [P] * 6 + [P, P, P, P, Z, P]
        L.moe_read_device_status.restype = I
        L.moe_read_device_status.argtypes = [P, P]
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


@functools.lru_cache(maxsize=1024)
def _shape_of(T, d, d_ff, E, k) -> MoeShape:
    return MoeShape(T, d, d_ff, E, k)


def _shape(shape) -> MoeShape:
    T, d, d_ff, E, k = map(int, shape)
    return _shape_of(T, d, d_ff, E, k)  # passed by value: one object serves a shape's calls


def _p(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without a Stream object around it (3 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def _check(fn: str, rc: int):
    if rc != MOE_OK:
        raise MoeError(fn, rc)


def _dev(t: torch.Tensor, name: str, dtype, shape=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _new(shape, dtype, like):
    return torch.empty(shape, dtype=dtype, device=like.device)


def moe_check_shape(shape) -> int:
    return lib().moe_check_shape(_shape(shape))


def moe_expert_workspace_bytes(shape) -> int:
    return lib().moe_expert_workspace_bytes(_shape(shape))


def moe_forward_workspace_bytes(shape) -> int:
    return lib().moe_forward_workspace_bytes(_shape(shape))


def moe_forward_kernel_count(shape) -> int:
    """Kernels one moe_forward of `shape` launches on the current device (5 or 6; 0 for
    T == 0); MoeError for a shape moe_forward rejects."""
    n = lib().moe_forward_kernel_count(_shape(shape))
    if n < 0:
        _check("moe_forward_kernel_count", -n)
    return n


def moe_forward_hostio_workspace_bytes(shape) -> int:
    return lib().moe_forward_hostio_workspace_bytes(_shape(shape))


def workspace(nbytes: int, device) -> torch.Tensor:
    """Device workspace of `nbytes` bytes (256-byte aligned by the caching allocator)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def moe_route(shape, x, Wg, bias=None, idx=None, gate=None, logits=None, want_logits=False,
              stream=None):
    T, d, d_ff, E, k = shape
    _dev(x, "x", torch.bfloat16, (T, d))
    _dev(Wg, "Wg", torch.bfloat16, (d, E))
    _dev(bias, "bias", torch.float32, (E,))
    idx = _new((T, k), torch.int32, x) if idx is None else idx
    gate = _new((T, k), torch.float32, x) if gate is None else gate
    if logits is None and want_logits:
        logits = _new((T, E), torch.float32, x)
    _dev(idx, "idx", torch.int32, (T, k))
    _dev(gate, "gate", torch.float32, (T, k))
    _dev(logits, "logits", torch.float32, (T, E))
    _check("moe_route", lib().moe_route(_shape(shape), _p(x), _p(Wg), _p(bias), _p(idx), _p(gate),
                                        _p(logits), _stream(stream)))
    return idx, gate, logits


def moe_dispatch(shape, idx, x, offsets=None, perm_tok=None, inv=None, x_sorted=None,
                 stream=None):
    T, d, d_ff, E, k = shape
    _dev(idx, "idx", torch.int32, (T, k))
    _dev(x, "x", torch.bfloat16, (T, d))
    offsets = _new((E + 1,), torch.int32, x) if offsets is None else offsets
    perm_tok = _new((T * k,), torch.int32, x) if perm_tok is None else perm_tok
    inv = _new((T, k), torch.int32, x) if inv is None else inv
    x_sorted = _new((T * k, d), torch.bfloat16, x) if x_sorted is None else x_sorted
    _dev(offsets, "offsets", torch.int32, (E + 1,))
    _dev(perm_tok, "perm_tok", torch.int32, (T * k,))
    _dev(inv, "inv", torch.int32, (T, k))
    _dev(x_sorted, "x_sorted", torch.bfloat16, (T * k, d))
    _check("moe_dispatch", lib().moe_dispatch(_shape(shape), _p(idx), _p(x), _p(offsets),
                                              _p(perm_tok), _p(inv), _p(x_sorted),
                                              _stream(stream)))
    return offsets, perm_tok, inv, x_sorted


def _expert_args(shape, x_sorted, offsets, W1, W3, W2, h, o, ws):
    T, d, d_ff, E, k = shape
    R = T * k
    _dev(x_sorted, "x_sorted", torch.bfloat16, (R, d))
    _dev(offsets, "offsets", torch.int32, (E + 1,))
    _dev(W1, "W1", torch.bfloat16, (E, d, d_ff))
    _dev(W3, "W3", torch.bfloat16, (E, d, d_ff))
    _dev(W2, "W2", torch.bfloat16, (E, d_ff, d))
    h = _new((R, d_ff), torch.bfloat16, x_sorted) if h is None else h
    o = _new((R, d), torch.float32, x_sorted) if o is None else o
    ws = workspace(moe_expert_workspace_bytes(shape), x_sorted.device) if ws is None else ws
    _dev(h, "h", torch.bfloat16, (R, d_ff))
    _dev(o, "o", torch.float32, (R, d))
    _dev(ws, "ws", torch.uint8)
    return h, o, ws


def moe_expert_swiglu(shape, x_sorted, offsets, W1, W3, W2, h=None, o=None, ws=None,
                      stream=None):
    h, o, ws = _expert_args(shape, x_sorted, offsets, W1, W3, W2, h, o, ws)
    _check("moe_expert_swiglu",
           lib().moe_expert_swiglu(_shape(shape), _p(x_sorted), _p(offsets), _p(W1), _p(W3),
                                   _p(W2), _p(h), _p(o), _p(ws), ws.numel(), _stream(stream)))
    return h, o, ws


def _expert_bias_args(shape, expert_bias):
    """(b1, b3, b2) float32 device tensors [E,d_ff], [E,d_ff], [E,d], each may be None."""
    T, d, d_ff, E, k = shape
    if expert_bias is None:
        return None, None, None
    b1, b3, b2 = expert_bias
    _dev(b1, "b1", torch.float32, (E, d_ff))
    _dev(b3, "b3", torch.float32, (E, d_ff))
    _dev(b2, "b2", torch.float32, (E, d))
    return b1, b3, b2


def moe_expert_swiglu_bias(shape, x_sorted, offsets, W1, W3, W2, expert_bias, h=None, o=None,
                           ws=None, stream=None):
    """moe_expert_swiglu with the expert Linear biases expert_bias = (b1, b3, b2)."""
    h, o, ws = _expert_args(shape, x_sorted, offsets, W1, W3, W2, h, o, ws)
    b1, b3, b2 = _expert_bias_args(shape, expert_bias)
    _check("moe_expert_swiglu_bias",
           lib().moe_expert_swiglu_bias(_shape(shape), _p(x_sorted), _p(offsets), _p(W1), _p(W3),
                                        _p(W2), _p(b1), _p(b3), _p(b2), _p(h), _p(o), _p(ws),
                                        ws.numel(), _stream(stream)))
    return h, o, ws


def moe_expert_swiglu_stall_test(shape, x_sorted, offsets, W1, W3, W2, stall_after: int,
                                 timeout_ns: int, h=None, o=None, ws=None, stream=None):
    h, o, ws = _expert_args(shape, x_sorted, offsets, W1, W3, W2, h, o, ws)
    _check("moe_expert_swiglu_stall_test",
           lib().moe_expert_swiglu_stall_test(_shape(shape), _p(x_sorted), _p(offsets), _p(W1),
                                              _p(W3), _p(W2), _p(h), _p(o), _p(ws), ws.numel(),
                                              int(stall_after), int(timeout_ns),
                                              _stream(stream)))
    return h, o, ws


def moe_combine(shape, o, inv, gate, y=None, stream=None):
    T, d, d_ff, E, k = shape
    _dev(o, "o", torch.float32, (T * k, d))
    _dev(inv, "inv", torch.int32, (T, k))
    _dev(gate, "gate", torch.float32, (T, k))
    y = _new((T, d), torch.bfloat16, o) if y is None else y
    _dev(y, "y", torch.bfloat16, (T, d))
    _check("moe_combine", lib().moe_combine(_shape(shape), _p(o), _p(inv), _p(gate), _p(y),
                                            _stream(stream)))
    return y


def moe_forward(shape, x, Wg, bias, W1, W3, W2, y=None, idx_out=None, gate_out=None, ws=None,
                stream=None):
    T, d, d_ff, E, k = shape
    _dev(x, "x", torch.bfloat16, (T, d))
    _dev(Wg, "Wg", torch.bfloat16, (d, E))
    _dev(bias, "bias", torch.float32, (E,))
    _dev(W1, "W1", torch.bfloat16, (E, d, d_ff))
    _dev(W3, "W3", torch.bfloat16, (E, d, d_ff))
    _dev(W2, "W2", torch.bfloat16, (E, d_ff, d))
    y = _new((T, d), torch.bfloat16, x) if y is None else y
    ws = workspace(moe_forward_workspace_bytes(shape), x.device) if ws is None else ws
    _dev(y, "y", torch.bfloat16, (T, d))
    _dev(idx_out, "idx_out", torch.int32, (T, k))
    _dev(gate_out, "gate_out", torch.float32, (T, k))
    _dev(ws, "ws", torch.uint8)
    _check("moe_forward", lib().moe_forward(_shape(shape), _p(x), _p(Wg), _p(bias), _p(W1), _p(W3),
                                            _p(W2), _p(y), _p(idx_out), _p(gate_out), _p(ws),
                                            ws.numel(), _stream(stream)))
    return y


def moe_forward_bias(shape, x, Wg, bias, W1, W3, W2, expert_bias, y=None, idx_out=None,
                     gate_out=None, ws=None, stream=None):
    """moe_forward with the expert Linear biases expert_bias = (b1, b3, b2)."""
    T, d, d_ff, E, k = shape
    _dev(x, "x", torch.bfloat16, (T, d))
    _dev(Wg, "Wg", torch.bfloat16, (d, E))
    _dev(bias, "bias", torch.float32, (E,))
    _dev(W1, "W1", torch.bfloat16, (E, d, d_ff))
    _dev(W3, "W3", torch.bfloat16, (E, d, d_ff))
    _dev(W2, "W2", torch.bfloat16, (E, d_ff, d))
    b1, b3, b2 = _expert_bias_args(shape, expert_bias)
    y = _new((T, d), torch.bfloat16, x) if y is None else y
    ws = workspace(moe_forward_workspace_bytes(shape), x.device) if ws is None else ws
    _dev(y, "y", torch.bfloat16, (T, d))
    _dev(idx_out, "idx_out", torch.int32, (T, k))
    _dev(gate_out, "gate_out", torch.float32, (T, k))
    _dev(ws, "ws", torch.uint8)
    _check("moe_forward_bias",
           lib().moe_forward_bias(_shape(shape), _p(x), _p(Wg), _p(bias), _p(W1), _p(W3), _p(W2),
                                  _p(b1), _p(b3), _p(b2), _p(y), _p(idx_out), _p(gate_out),
                                  _p(ws), ws.numel(), _stream(stream)))
    return y


PROFILE_EVENTS = ("start", "router", "dispatch_index", "dispatch_scatter", "gemm1_swiglu",
                  "gemm2_down", "combine")


def moe_forward_profiled(shape, x, Wg, bias, W1, W3, W2, events, y=None, ws=None, stream=None):
    """moe_forward that records the 7 torch.cuda.Event objects in `events` between its
    launches (see PROFILE_EVENTS); the events must have been recorded once already so
    that their CUDA handles exist."""
    T, d, d_ff, E, k = shape
    _dev(x, "x", torch.bfloat16, (T, d))
    _dev(Wg, "Wg", torch.bfloat16, (d, E))
    _dev(bias, "bias", torch.float32, (E,))
    _dev(W1, "W1", torch.bfloat16, (E, d, d_ff))
    _dev(W3, "W3", torch.bfloat16, (E, d, d_ff))
    _dev(W2, "W2", torch.bfloat16, (E, d_ff, d))
    y = _new((T, d), torch.bfloat16, x) if y is None else y
    ws = workspace(moe_forward_workspace_bytes(shape), x.device) if ws is None else ws
    _dev(y, "y", torch.bfloat16, (T, d))
    _dev(ws, "ws", torch.uint8)
    if len(events) != len(PROFILE_EVENTS):
        raise ValueError(f"need {len(PROFILE_EVENTS)} events")
    handles = (ctypes.c_void_p * len(events))(*[ev.cuda_event for ev in events])
    _check("moe_forward_profiled",
           lib().moe_forward_profiled(_shape(shape), _p(x), _p(Wg), _p(bias), _p(W1), _p(W3),
                                      _p(W2), _p(y), _p(ws), ws.numel(), handles, len(events),
                                      _stream(stream)))
    return y


def moe_forward_hostio(shape, x_host, Wg, bias, W1, W3, W2, y_host, ws, stream=None):
    """x_host / y_host: CPU bf16 tensors (pinned for asynchronous copies)."""
    T, d, d_ff, E, k = shape
    for name, t in (("x_host", x_host), ("y_host", y_host)):
        if t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() \
                or tuple(t.shape) != (T, d):
            raise ValueError(f"{name} must be a contiguous CPU bf16 tensor of shape {(T, d)}")
    _dev(Wg, "Wg", torch.bfloat16, (d, E))
    _dev(bias, "bias", torch.float32, (E,))
    _dev(W1, "W1", torch.bfloat16, (E, d, d_ff))
    _dev(W3, "W3", torch.bfloat16, (E, d, d_ff))
    _dev(W2, "W2", torch.bfloat16, (E, d_ff, d))
    _dev(ws, "ws", torch.uint8)
    _check("moe_forward_hostio",
           lib().moe_forward_hostio(_shape(shape), _p(x_host), _p(Wg), _p(bias), _p(W1), _p(W3),
                                    _p(W2), _p(y_host), _p(ws), ws.numel(), _stream(stream)))
    return y_host


def moe_forward_hostio_batches_workspace_bytes(shape) -> int:
    return lib().moe_forward_hostio_batches_workspace_bytes(_shape(shape))


def moe_forward_hostio_batches(shape, xs_host, Wg, bias, W1, W3, W2, ys_host, ws, stream=None):
    """xs_host / ys_host: equal-length sequences of CPU bf16 tensors of shape (T, d)
    (pinned for asynchronous copies); batch b reads xs_host[b] and writes ys_host[b]."""
    T, d, d_ff, E, k = shape
    if len(xs_host) != len(ys_host) or len(xs_host) < 1:
        raise ValueError("xs_host and ys_host must be non-empty and of equal length")
    for name, seq in (("xs_host", xs_host), ("ys_host", ys_host)):
        for t in seq:
            if t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() \
                    or tuple(t.shape) != (T, d):
                raise ValueError(f"every {name} entry must be a contiguous CPU bf16 tensor "
                                 f"of shape {(T, d)}")
    _dev(Wg, "Wg", torch.bfloat16, (d, E))
    _dev(bias, "bias", torch.float32, (E,))
    _dev(W1, "W1", torch.bfloat16, (E, d, d_ff))
    _dev(W3, "W3", torch.bfloat16, (E, d, d_ff))
    _dev(W2, "W2", torch.bfloat16, (E, d_ff, d))
    _dev(ws, "ws", torch.uint8)
    n = len(xs_host)
    xp = (ctypes.c_void_p * n)(*[t.data_ptr() for t in xs_host])
    yp = (ctypes.c_void_p * n)(*[t.data_ptr() for t in ys_host])
    _check("moe_forward_hostio_batches",
           lib().moe_forward_hostio_batches(_shape(shape), n, ctypes.cast(xp, ctypes.c_void_p),
                                            _p(Wg), _p(bias), _p(W1), _p(W3), _p(W2),
                                            ctypes.cast(yp, ctypes.c_void_p), _p(ws), ws.numel(),
                                            _stream(stream)))
    return ys_host


def _host_batches(shape, xs_host, ys_host):
    T, d, d_ff, E, k = shape
    if len(xs_host) != len(ys_host) or len(xs_host) < 1:
        raise ValueError("xs_host and ys_host must be non-empty and of equal length")
    for name, seq in (("xs_host", xs_host), ("ys_host", ys_host)):
        for t in seq:
            if t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() \
                    or tuple(t.shape) != (T, d):
                raise ValueError(f"every {name} entry must be a contiguous CPU bf16 tensor "
                                 f"of shape {(T, d)}")
    n = len(xs_host)
    xp = (ctypes.c_void_p * n)(*[t.data_ptr() for t in xs_host])
    yp = (ctypes.c_void_p * n)(*[t.data_ptr() for t in ys_host])
    return n, xp, yp


def moe_forward_hostio_batches_stall_test(shape, xs_host, Wg, bias, W1, W3, W2, ys_host, ws,
                                          stall_batch: int, stall_after: int, timeout_ns: int,
                                          stream=None):
    """moe_forward_hostio_batches with the expert producer of batch `stall_batch`
    stopping after `stall_after` stages and that batch's waits bounded by
    `timeout_ns` (test of the error path of the queue)."""
    T, d, d_ff, E, k = shape
    n, xp, yp = _host_batches(shape, xs_host, ys_host)
    _dev(Wg, "Wg", torch.bfloat16, (d, E))
    _dev(bias, "bias", torch.float32, (E,))
    _dev(W1, "W1", torch.bfloat16, (E, d, d_ff))
    _dev(W3, "W3", torch.bfloat16, (E, d, d_ff))
    _dev(W2, "W2", torch.bfloat16, (E, d_ff, d))
    _dev(ws, "ws", torch.uint8)
    _check("moe_forward_hostio_batches_stall_test",
           lib().moe_forward_hostio_batches_stall_test(
               _shape(shape), n, ctypes.cast(xp, ctypes.c_void_p), _p(Wg), _p(bias), _p(W1),
               _p(W3), _p(W2), ctypes.cast(yp, ctypes.c_void_p), _p(ws), ws.numel(),
               int(stall_batch), int(stall_after), int(timeout_ns), _stream(stream)))
    return ys_host


def moe_forward_hostio_stall_test(shape, x_host, Wg, bias, W1, W3, W2, y_host, ws,
                                  stall_chunk: int, stall_after: int, timeout_ns: int,
                                  stream=None):
    """moe_forward_hostio with the expert producer of token chunk `stall_chunk`
    stopping after `stall_after` stages and that chunk's waits bounded by
    `timeout_ns` (test of the error path of the chunked pipeline)."""
    T, d, d_ff, E, k = shape
    for name, t in (("x_host", x_host), ("y_host", y_host)):
        if t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() \
                or tuple(t.shape) != (T, d):
            raise ValueError(f"{name} must be a contiguous CPU bf16 tensor of shape {(T, d)}")
    _dev(Wg, "Wg", torch.bfloat16, (d, E))
    _dev(bias, "bias", torch.float32, (E,))
    _dev(W1, "W1", torch.bfloat16, (E, d, d_ff))
    _dev(W3, "W3", torch.bfloat16, (E, d, d_ff))
    _dev(W2, "W2", torch.bfloat16, (E, d_ff, d))
    _dev(ws, "ws", torch.uint8)
    _check("moe_forward_hostio_stall_test",
           lib().moe_forward_hostio_stall_test(_shape(shape), _p(x_host), _p(Wg), _p(bias), _p(W1),
                                               _p(W3), _p(W2), _p(y_host), _p(ws), ws.numel(),
                                               int(stall_chunk), int(stall_after),
                                               int(timeout_ns), _stream(stream)))
    return y_host


def moe_forward_static(shape, x, Wg, bias, W1, W3, W2, y=None, device_status=None, stream=None):
    """moe_forward without a workspace argument: the library's fixed 8 MiB device
    scratch array stands in for it (for callers that cannot allocate device memory).
    `device_status`: optional CUDA int32 tensor of one element that receives the
    call's status word."""
    T, d, d_ff, E, k = shape
    _dev(x, "x", torch.bfloat16, (T, d))
    _dev(Wg, "Wg", torch.bfloat16, (d, E))
    _dev(bias, "bias", torch.float32, (E,))
    _dev(W1, "W1", torch.bfloat16, (E, d, d_ff))
    _dev(W3, "W3", torch.bfloat16, (E, d, d_ff))
    _dev(W2, "W2", torch.bfloat16, (E, d_ff, d))
    y = _new((T, d), torch.bfloat16, x) if y is None else y
    _dev(y, "y", torch.bfloat16, (T, d))
    _dev(device_status, "device_status", torch.int32, (1,))
    _check("moe_forward_static",
           lib().moe_forward_static(_shape(shape), _p(x), _p(Wg), _p(bias), _p(W1), _p(W3),
                                    _p(W2), _p(y), _p(device_status), _stream(stream)))
    return y


def moe_block_workspace_bytes(shape) -> int:
    return lib().moe_block_workspace_bytes(_shape(shape))


def moe_block_forward(shape, U, gamma, Wg, bias, W1, W3, W2, eps=1e-5, H=None, ws=None,
                      stream=None):
    """H = U + MoE(RMSNorm(U)) through moe_block_forward."""
    T, d, d_ff, E, k = shape
    _dev(U, "U", torch.bfloat16, (T, d))
    _dev(gamma, "gamma", torch.bfloat16, (d,))
    _dev(Wg, "Wg", torch.bfloat16, (d, E))
    _dev(bias, "bias", torch.float32, (E,))
    _dev(W1, "W1", torch.bfloat16, (E, d, d_ff))
    _dev(W3, "W3", torch.bfloat16, (E, d, d_ff))
    _dev(W2, "W2", torch.bfloat16, (E, d_ff, d))
    H = _new((T, d), torch.bfloat16, U) if H is None else H
    ws = workspace(moe_block_workspace_bytes(shape), U.device) if ws is None else ws
    _dev(H, "H", torch.bfloat16, (T, d))
    _dev(ws, "ws", torch.uint8)
    _check("moe_block_forward",
           lib().moe_block_forward(_shape(shape), _p(U), _p(gamma), float(eps), _p(Wg), _p(bias),
                                   _p(W1), _p(W3), _p(W2), _p(H), _p(ws), ws.numel(),
                                   _stream(stream)))
    return H


def moe_aux_loss(shape, logits, idx, mask=None, want_stats=False, stream=None):
    """Load-balancing term E * sum_s sum_i f_{s,i} P_i.  Returns (aux [1], f [k,E] or None,
    P [E] or None) as CUDA float32 tensors.  shape's T is the number of rows of logits."""
    T, d, d_ff, E, k = shape
    _dev(logits, "logits", torch.float32, (T, E))
    _dev(idx, "idx", torch.int32, (T, k))
    _dev(mask, "mask", torch.uint8, (T,))
    aux = _new((1,), torch.float32, logits)
    f = _new((k, E), torch.float32, logits) if want_stats else None
    P = _new((E,), torch.float32, logits) if want_stats else None
    _check("moe_aux_loss", lib().moe_aux_loss(_shape(shape), _p(logits), _p(idx), _p(mask), _p(aux),
                                              _p(f), _p(P), _stream(stream)))
    return aux, f, P


def moe_read_device_status(ws, stream=None) -> int:
    """Synchronises the stream and returns the status word of `ws` (MOE_OK or an error code)."""
    return lib().moe_read_device_status(_p(ws), _stream(stream))


# ------------------------------------------------------------------ scored routing, int8 experts

_LOGITS_TYPES = {torch.float32: 0, torch.bfloat16: 1}


def _arg(t, name: str, dtype, shape, device: int):
    """The pointer of a checked argument (None stays None): _dev's checks, and that it lies on
    the current device, on whose stream the work is enqueued."""
    if t is None:
        return None
    if t.is_cuda and t.dtype == dtype and t.shape == shape and t.is_contiguous() \
            and t.get_device() == device:
        return t.data_ptr()
    _dev(t, name, dtype, shape)
    raise ValueError(f"{name} is on {t.device}, the current device is cuda:{device}")


def _given(t, name: str, like):
    """A required argument; `like`: what says where new outputs go."""
    if t is None:
        raise ValueError(f"{name} is required")
    if not like.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _queue(stream, device: int):
    """The handle of `stream`, of the current device, or of its current stream."""
    if stream is None:
        return _stream(None) if _raw_stream is None else _raw_stream(device)
    if stream.device_index != device:
        raise ValueError(f"stream is of cuda:{stream.device_index}, "
                         f"the current device is cuda:{device}")
    return stream.cuda_stream


def _empty(shape, dtype, like, stream):
    """A new tensor of the stream that the work runs on, so that its memory is neither still in use
    by another stream's work nor, once released, handed out before this work is done."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _out(t, name: str, dtype, shape, like, stream, device: int):
    """An output and its pointer: the caller's, checked, or a new one."""
    if t is None:
        t = _empty(shape, dtype, like, stream)
        return t, t.data_ptr()
    return t, _arg(t, name, dtype, shape, device)


def _scratch(nbytes: int, like, stream):
    return _empty((max(nbytes, 256),), torch.uint8, like, stream)


def _logits(t, shape, device: int):
    """(pointer, type code) of router logits."""
    kind = _LOGITS_TYPES.get(t.dtype)
    if kind is None:
        raise ValueError(f"logits must be float32 or bfloat16, got {t.dtype}")
    return _arg(t, "logits", t.dtype, (shape[0], shape[3]), device), kind


def moe_check_scoring(shape, scoring: MoeScoring) -> int:
    return lib().moe_check_scoring(_shape(shape), scoring)


def moe_check_shape_int8(shape) -> int:
    return lib().moe_check_shape_int8(_shape(shape))


def moe_expert_swiglu_int8_workspace_bytes(shape) -> int:
    return lib().moe_expert_swiglu_int8_workspace_bytes(_shape(shape))


def moe_forward_int8_workspace_bytes(shape) -> int:
    return lib().moe_forward_int8_workspace_bytes(_shape(shape))


def moe_route_scored(shape, logits, scoring: MoeScoring, bias=None, mask=None, idx=None, gate=None,
                     stream=None):
    """Experts and gates of each token from its router logits [T, E] (float32 or bfloat16).

    `bias` [E] float32 steers the selection only; rows whose `mask` [T] uint8 is 0 get no expert.
    Returns (idx [T, k] int32, gate [T, k] float32); idx -1 (gate 0) marks a slot that
    no expert fills.  Only T, E and k of `shape` are used.  Like every call here it gives plain values:
    logits that require a gradient give gates without a graph, and moe_route_scored_backward is
    called with their gradient."""
    T, d, d_ff, E, k = shape
    _given(logits, "logits", logits)
    dev = torch.cuda.current_device()
    lp, kind = _logits(logits, shape, dev)
    bp = _arg(bias, "bias", torch.float32, (E,), dev)
    mp = _arg(mask, "mask", torch.uint8, (T,), dev)
    idx, ip = _out(idx, "idx", torch.int32, (T, k), logits, stream, dev)
    gate, gp = _out(gate, "gate", torch.float32, (T, k), logits, stream, dev)
    _check("moe_route_scored",
           lib().moe_route_scored(_shape(shape), scoring, lp, kind, bp, mp, ip, gp,
                                  _queue(stream, dev)))
    return idx, gate


def moe_route_scored_backward(shape, logits, scoring: MoeScoring, idx, dgate, dlogits=None,
                              stream=None):
    """Gradient of moe_route_scored's gates to the logits, in the logits' type.

    `idx` is the forward call's; `dgate` [T, k] float32 the gates' gradient, which the caller forms
    (for a training step around these calls: nothing in this package does)."""
    T, d, d_ff, E, k = shape
    _given(logits, "logits", logits)
    dev = torch.cuda.current_device()
    lp, kind = _logits(logits, shape, dev)
    ip = _arg(idx, "idx", torch.int32, (T, k), dev)
    gp = _arg(dgate, "dgate", torch.float32, (T, k), dev)
    dlogits, dp = _out(dlogits, "dlogits", logits.dtype, (T, E), logits, stream, dev)
    _check("moe_route_scored_backward",
           lib().moe_route_scored_backward(_shape(shape), scoring, lp, kind, ip, gp, dp,
                                           _queue(stream, dev)))
    return dlogits


def moe_quantize_weights_int8(W, Wq=None, scale=None, stream=None):
    """(Wq [E, N, K] int8, scale [E, N] float32) of bf16 weights W [E, K, N]: one scale for
    each output channel.  The pairs are what moe_expert_swiglu_int8 takes as W1, W3, W2."""
    _given(W, "W", W)
    if W.dim() != 3:
        raise ValueError(f"W must have shape (E, K, N), got {tuple(W.shape)}")
    E, K, N = W.shape
    dev = torch.cuda.current_device()
    wp = _arg(W, "W", torch.bfloat16, (E, K, N), dev)
    Wq, qp = _out(Wq, "Wq", torch.int8, (E, N, K), W, stream, dev)
    scale, sp = _out(scale, "scale", torch.float32, (E, N), W, stream, dev)
    _check("moe_quantize_weights_int8",
           lib().moe_quantize_weights_int8(E, K, N, wp, qp, sp, _queue(stream, dev)))
    return Wq, scale


def moe_dispatch_int8(shape, idx, x, offsets=None, perm_tok=None, inv=None, xq=None, xs=None,
                      stream=None):
    """moe_dispatch whose sorted rows leave quantised: returns (offsets, perm_tok, inv,
    xq [T*k, d] int8, xs [T*k] float32)."""
    T, d, d_ff, E, k = shape
    _given(x, "x", x)
    dev = torch.cuda.current_device()
    ip = _arg(idx, "idx", torch.int32, (T, k), dev)
    xp = _arg(x, "x", torch.bfloat16, (T, d), dev)
    offsets, op = _out(offsets, "offsets", torch.int32, (E + 1,), x, stream, dev)
    perm_tok, pp = _out(perm_tok, "perm_tok", torch.int32, (T * k,), x, stream, dev)
    inv, vp = _out(inv, "inv", torch.int32, (T, k), x, stream, dev)
    xq, qp = _out(xq, "xq", torch.int8, (T * k, d), x, stream, dev)
    xs, sp = _out(xs, "xs", torch.float32, (T * k,), x, stream, dev)
    _check("moe_dispatch_int8",
           lib().moe_dispatch_int8(_shape(shape), ip, xp, op, pp, vp, qp, sp, _queue(stream, dev)))
    return offsets, perm_tok, inv, xq, xs


def _int8_weights(shape, W1, W3, W2, device: int):
    """Pointers of the (int8, scale) pairs W1, W3 [E, d_ff, d] and W2 [E, d, d_ff]."""
    T, d, d_ff, E, k = shape
    (q1, s1), (q3, s3), (q2, s2) = W1, W3, W2
    return (_arg(q1, "W1", torch.int8, (E, d_ff, d), device),
            _arg(s1, "W1 scale", torch.float32, (E, d_ff), device),
            _arg(q3, "W3", torch.int8, (E, d_ff, d), device),
            _arg(s3, "W3 scale", torch.float32, (E, d_ff), device),
            _arg(q2, "W2", torch.int8, (E, d, d_ff), device),
            _arg(s2, "W2 scale", torch.float32, (E, d), device))


def _ws_arg(ws, device: int):
    """(pointer, bytes) of a workspace: a uint8 tensor of any length."""
    return _arg(ws, "ws", torch.uint8, ws.shape, device), ws.numel()


def _int8_expert_args(shape, xq, xs, offsets, W1, W3, W2, o, ws, stream):
    T, d, d_ff, E, k = shape
    R = T * k
    _given(xq, "xq", xq)
    dev = torch.cuda.current_device()
    o, op = _out(o, "o", torch.bfloat16, (R, d), xq, stream, dev)
    if ws is None:
        ws = _scratch(moe_expert_swiglu_int8_workspace_bytes(shape), xq, stream)
    args = (_arg(xq, "xq", torch.int8, (R, d), dev), _arg(xs, "xs", torch.float32, (R,), dev),
            _arg(offsets, "offsets", torch.int32, (E + 1,), dev),
            *_int8_weights(shape, W1, W3, W2, dev), op, *_ws_arg(ws, dev))
    return args, o, ws


def moe_expert_swiglu_int8(shape, xq, xs, offsets, W1, W3, W2, o=None, ws=None, stream=None):
    """The SwiGLU experts in 8-bit integers over the rows of moe_dispatch_int8.

    W1, W3, W2 are the (int8, scale) pairs of moe_quantize_weights_int8.  Returns
    (o [T*k, d] bfloat16, ws)."""
    args, o, ws = _int8_expert_args(shape, xq, xs, offsets, W1, W3, W2, o, ws, stream)
    _check("moe_expert_swiglu_int8",
           lib().moe_expert_swiglu_int8(_shape(shape), *args, _queue(stream, xq.get_device())))
    return o, ws


def moe_expert_swiglu_int8_stall_test(shape, xq, xs, offsets, W1, W3, W2, stall_after: int,
                                      timeout_ns: int, o=None, ws=None, stream=None):
    args, o, ws = _int8_expert_args(shape, xq, xs, offsets, W1, W3, W2, o, ws, stream)
    _check("moe_expert_swiglu_int8_stall_test",
           lib().moe_expert_swiglu_int8_stall_test(_shape(shape), *args, int(stall_after),
                                                   int(timeout_ns),
                                                   _queue(stream, xq.get_device())))
    return o, ws


def moe_combine_bf16(shape, o, inv, gate, y=None, stream=None):
    """moe_combine over bfloat16 expert outputs o [T*k, d]."""
    T, d, d_ff, E, k = shape
    _given(o, "o", o)
    dev = torch.cuda.current_device()
    y, yp = _out(y, "y", torch.bfloat16, (T, d), o, stream, dev)
    _check("moe_combine_bf16",
           lib().moe_combine_bf16(_shape(shape), _arg(o, "o", torch.bfloat16, (T * k, d), dev),
                                  _arg(inv, "inv", torch.int32, (T, k), dev),
                                  _arg(gate, "gate", torch.float32, (T, k), dev),
                                  yp, _queue(stream, dev)))
    return y


def moe_forward_int8(shape, x, logits, scoring: MoeScoring, W1, W3, W2, route_bias=None, mask=None,
                     y=None, idx_out=None, gate_out=None, ws=None, stream=None):
    """The layer with scored routing and int8 experts, from tokens x [T, d] bfloat16 and router
    logits [T, E] (float32, as of moe_route, or bfloat16).  W1, W3, W2 are the
    (int8, scale) pairs of moe_quantize_weights_int8."""
    T, d, d_ff, E, k = shape
    _given(x, "x", x)
    _given(logits, "logits", logits)
    dev = torch.cuda.current_device()
    lp, kind = _logits(logits, shape, dev)
    y, yp = _out(y, "y", torch.bfloat16, (T, d), x, stream, dev)
    ws = _scratch(moe_forward_int8_workspace_bytes(shape), x, stream) if ws is None else ws
    _check("moe_forward_int8",
           lib().moe_forward_int8(_shape(shape), _arg(x, "x", torch.bfloat16, (T, d), dev), lp, kind,
                                  scoring, _arg(route_bias, "route_bias", torch.float32, (E,), dev),
                                  _arg(mask, "mask", torch.uint8, (T,), dev),
                                  *_int8_weights(shape, W1, W3, W2, dev),
                                  yp, _arg(idx_out, "idx_out", torch.int32, (T, k), dev),
                                  _arg(gate_out, "gate_out", torch.float32, (T, k), dev),
                                  *_ws_arg(ws, dev), _queue(stream, dev)))
    return y
