"""Python binding of libmoe.so, the MI355X (gfx950) sparse-MoE layer forward.

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  Functions carry the C entry points' names (see include/moe.h for
the full contract) and take torch tensors that live on the current HIP
device; PyTorch provides the device memory and the stream, nothing else.

The library must have been built (``__graft_entry__.build()`` or
``python -m sparse_moe_layer_fp32_amd._build``); importing fails loudly
otherwise -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import dataclasses
import itertools
import math
import operator
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = range(5)
STAGES = ("router_gemm", "topk", "rank", "scan", "scatter", "gateup", "down", "combine")
MOE_NUM_STAGES = len(STAGES)
(MOE_WS_TOPK_IDS, MOE_WS_TOPK_W, MOE_WS_EXPERT_OFFSETS, MOE_WS_SORTED_PAIRS, MOE_WS_PAIR_POS,
 MOE_WS_H, MOE_WS_O, MOE_WS_FUSED_CTL, MOE_WS_FUSED_STATUS) = range(9)
FUSED_MAX_TOKENS, FUSED_MAX_PAIRS = 256, 2048


class MoeError(RuntimeError):
    def __init__(self, status: int, text: str):
        super().__init__(f"moe status {status}: {text}")
        self.status = status


class moe_config(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("hidden", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("inter", ctypes.c_int32), ("inter_shared", ctypes.c_int32),
                ("routed_scaling", ctypes.c_float), ("renormalize", ctypes.c_int32),
                ("swiglu_limit", ctypes.c_float), ("swiglu_limit_shared", ctypes.c_float)]


def make_config(tokens, hidden=4096, num_experts=288, top_k=8, inter=1280, inter_shared=1280,
                routed_scaling=3.0, renormalize=True, swiglu_limit=0.0,
                swiglu_limit_shared=0.0) -> moe_config:
    return moe_config(int(tokens), int(hidden), int(num_experts), int(top_k), int(inter),
                      int(inter_shared), float(routed_scaling), int(bool(renormalize)),
                      float(swiglu_limit), float(swiglu_limit_shared))


class moe_dense_config(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("swiglu_limit", ctypes.c_float), ("reserved", ctypes.c_int32)]


def make_dense_config(tokens, hidden=4096, inter=11264, swiglu_limit=0.0) -> moe_dense_config:
    return moe_dense_config(int(tokens), int(hidden), int(inter), float(swiglu_limit), 0)


ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")  # MOE_ACT_*
DTYPES = ("bf16", "f32")                                      # MOE_DTYPE_*


def _index(names, value, what):
    if value not in names:
        raise ValueError(f"{what} {value!r} is none of {', '.join(names)}")
    return names.index(value)


class moe_linear_config(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("in_features", ctypes.c_int32),
                ("out_features", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("dw_dtype", ctypes.c_int32),
                ("accumulate", ctypes.c_int32)]


def make_linear_config(tokens, in_features, out_features, activation="none", y_dtype="bf16",
                       dw_dtype="f32", accumulate=False) -> moe_linear_config:
    return moe_linear_config(int(tokens), int(in_features), int(out_features),
                             _index(ACTIVATIONS, activation, "activation"),
                             _index(DTYPES, y_dtype, "y_dtype"),
                             _index(DTYPES, dw_dtype, "dw_dtype"), int(bool(accumulate)))


class moe_grouped_config(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("x_rows", ctypes.c_int64),
                ("num_groups", ctypes.c_int32), ("in_features", ctypes.c_int32),
                ("out_features", ctypes.c_int32), ("row_div", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("dw_dtype", ctypes.c_int32),
                ("accumulate", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def make_grouped_config(rows, num_groups, in_features, out_features, x_rows=None, row_div=1,
                        y_dtype="bf16", dw_dtype="f32", accumulate=False) -> moe_grouped_config:
    """x_rows: rows of x when row_ids is passed (default: rows)."""
    return moe_grouped_config(int(rows), int(rows if x_rows is None else x_rows), int(num_groups),
                              int(in_features), int(out_features), int(row_div),
                              _index(DTYPES, y_dtype, "y_dtype"),
                              _index(DTYPES, dw_dtype, "dw_dtype"), int(bool(accumulate)), 0)


class moe_swiglu_config(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("inter", ctypes.c_int32), ("ld", ctypes.c_int32),
                ("limit", ctypes.c_float), ("reserved", ctypes.c_int32)]


def make_swiglu_config(rows, inter, ld=0, limit=0.0) -> moe_swiglu_config:
    """ld: row stride of gate, up and their gradients (0: inter)."""
    return moe_swiglu_config(int(rows), int(inter), int(ld), float(limit), 0)


class moe_dispatch_config(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("rows", ctypes.c_int64), ("top_k", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("token_dtype", ctypes.c_int32),
                ("row_dtype", ctypes.c_int32)]


def make_dispatch_config(tokens, rows, top_k, hidden, token_dtype="bf16",
                         row_dtype="bf16") -> moe_dispatch_config:
    """rows: rows of the experts' side (tokens * top_k when every pair has one)."""
    return moe_dispatch_config(int(tokens), int(rows), int(top_k), int(hidden),
                               _index(DTYPES, token_dtype, "token_dtype"),
                               _index(DTYPES, row_dtype, "row_dtype"))


class moe_quantize_config(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("rows", ctypes.c_int64), ("top_k", ctypes.c_int32),
                ("features", ctypes.c_int32)]


def make_quantize_config(tokens, features, rows=None, top_k=1) -> moe_quantize_config:
    """rows: rows of the codes (default: tokens)."""
    return moe_quantize_config(int(tokens), int(tokens if rows is None else rows), int(top_k),
                               int(features))


_lib = None


def load_library():
    """Load libmoe.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it first "
                          "(python -m sparse_moe_layer_fp32_amd._build)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, cp = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(moe_config)
    lib.moe_workspace_size.argtypes = [cp]
    lib.moe_workspace_size.restype = sz
    lib.moe_last_error.argtypes = []
    lib.moe_last_error.restype = ctypes.c_char_p
    lib.moe_route.argtypes = [cp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_permute.argtypes = [cp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_forward.argtypes = [cp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_forward_timed.argtypes = lib.moe_forward.argtypes + [ctypes.POINTER(vp), ctypes.c_int]
    lib.moe_forward_noalloc.argtypes = [cp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.moe_workspace_view.argtypes = [cp, ctypes.c_int, ctypes.POINTER(sz), ctypes.POINTER(sz)]
    lib.moe_forward_fp8.argtypes = [cp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                    vp, sz, vp]
    dp = ctypes.POINTER(moe_dense_config)
    lib.moe_dense_workspace_size.argtypes = [dp]
    lib.moe_dense_workspace_size.restype = sz
    lib.moe_dense_forward.argtypes = [dp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_forward_fused.argtypes = lib.moe_forward.argtypes
    lp, gp, sp = (ctypes.POINTER(t) for t in (moe_linear_config, moe_grouped_config,
                                              moe_swiglu_config))
    lib.moe_linear_workspace_size.argtypes = [lp]
    lib.moe_linear_workspace_size.restype = sz
    lib.moe_linear_forward.argtypes = [lp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_linear_backward.argtypes = [lp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_grouped_workspace_size.argtypes = [gp]
    lib.moe_grouped_workspace_size.restype = sz
    lib.moe_grouped_forward.argtypes = [gp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_grouped_backward.argtypes = [gp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_swiglu_forward.argtypes = [sp, vp, vp, vp, vp]
    lib.moe_swiglu_backward.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp]
    rp, qp = ctypes.POINTER(moe_dispatch_config), ctypes.POINTER(moe_quantize_config)
    lib.moe_dispatch_forward.argtypes = [rp, vp, vp, vp, vp]
    lib.moe_dispatch_backward.argtypes = [rp, vp, vp, vp, vp, vp]
    lib.moe_combine_forward.argtypes = [rp, vp, vp, vp, vp, vp, vp]
    lib.moe_combine_backward.argtypes = [rp, vp, vp, vp, vp, vp, vp, vp]
    lib.moe_quantize_rows.argtypes = [qp, vp, vp, vp, vp, vp]
    lib.moe_quantize_weight.argtypes = [ctypes.c_int32] * 3 + [vp, vp, vp, vp]
    lib.moe_linear_fp8_workspace_size.argtypes = [lp]
    lib.moe_linear_fp8_workspace_size.restype = sz
    lib.moe_linear_forward_fp8.argtypes = [lp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_grouped_fp8_workspace_size.argtypes = [gp]
    lib.moe_grouped_fp8_workspace_size.restype = sz
    lib.moe_grouped_forward_fp8.argtypes = [gp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    for f in ("moe_route", "moe_permute", "moe_forward", "moe_forward_timed",
              "moe_workspace_view", "moe_dense_forward", "moe_forward_fp8", "moe_forward_fused",
              "moe_linear_forward", "moe_linear_backward", "moe_grouped_forward",
              "moe_grouped_backward", "moe_swiglu_forward", "moe_swiglu_backward",
              "moe_dispatch_forward", "moe_dispatch_backward", "moe_combine_forward",
              "moe_combine_backward", "moe_quantize_rows", "moe_quantize_weight",
              "moe_linear_forward_fp8", "moe_grouped_forward_fp8"):
        getattr(lib, f).restype = ctypes.c_int
    _lib = lib
    return lib


EXPORTED = ("moe_workspace_size", "moe_last_error", "moe_route", "moe_permute", "moe_forward",
            "moe_forward_timed", "moe_workspace_view", "moe_dense_workspace_size",
            "moe_dense_forward", "moe_forward_fp8", "moe_forward_fused",
            "moe_forward_noalloc", "moe_linear_workspace_size", "moe_linear_forward",
            "moe_linear_backward", "moe_grouped_workspace_size", "moe_grouped_forward",
            "moe_grouped_backward", "moe_swiglu_forward", "moe_swiglu_backward",
            "moe_dispatch_forward", "moe_dispatch_backward", "moe_combine_forward",
            "moe_combine_backward", "moe_quantize_rows", "moe_quantize_weight",
            "moe_linear_fp8_workspace_size", "moe_linear_forward_fp8",
            "moe_grouped_fp8_workspace_size", "moe_grouped_forward_fp8")
NOALLOC_SCRATCH_BYTES = 64 << 20  # MOE_NOALLOC_SCRATCH_BYTES


# ------------------------------------------------------------------ helpers

def _torch():
    import torch
    return torch


def _ptr(t, dtype=None, name="tensor", optional=False):
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on the GPU, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtype}")
    return t.data_ptr()


def _bf16():
    torch = _torch()
    return (torch.bfloat16, torch.uint16, torch.int16)


def _f32():
    return (_torch().float32,)


def _i32():
    return (_torch().int32,)


def _stream(stream):
    if stream is None:
        return _torch().cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int):
    if status != MOE_OK:
        raise MoeError(status, load_library().moe_last_error().decode())


def moe_last_error() -> str:
    return load_library().moe_last_error().decode()


def moe_workspace_size(cfg: moe_config) -> int:
    n = load_library().moe_workspace_size(ctypes.byref(cfg))
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, moe_last_error())
    return int(n)


def alloc_workspace(cfg: moe_config, device=None):
    """A zero-filled uint8 device tensor of moe_workspace_size(cfg) bytes
    (zero-filled once, as moe_forward_fused requires of its control words)."""
    torch = _torch()
    return torch.zeros(moe_workspace_size(cfg), dtype=torch.uint8,
                       device=device or torch.device("cuda"))


def moe_route(cfg, x, router_w, router_bias, topk_ids, topk_w, ws, stream=None):
    lib = load_library()
    _check(lib.moe_route(ctypes.byref(cfg), _ptr(x, _bf16(), "x"), _ptr(router_w, _f32(), "router_w"),
                         _ptr(router_bias, _f32(), "router_bias", True),
                         _ptr(topk_ids, _i32(), "topk_ids"), _ptr(topk_w, _f32(), "topk_w"),
                         _ptr(ws, None, "ws"), ws.numel() * ws.element_size(), _stream(stream)))


def moe_permute(cfg, topk_ids, expert_offsets, sorted_pairs, pair_pos, ws, stream=None):
    lib = load_library()
    _check(lib.moe_permute(ctypes.byref(cfg), _ptr(topk_ids, _i32(), "topk_ids"),
                           _ptr(expert_offsets, _i32(), "expert_offsets"),
                           _ptr(sorted_pairs, _i32(), "sorted_pairs"),
                           _ptr(pair_pos, _i32(), "pair_pos"), _ptr(ws, None, "ws"),
                           ws.numel() * ws.element_size(), _stream(stream)))


def _forward_args(cfg, x, router_w, router_bias, w_gate, w_up, w_down, ws_gate, ws_up, ws_down,
                  y, topk_ids_out, topk_w_out, ws, stream, no_ws=False):
    bf = _bf16()
    args = [ctypes.byref(cfg), _ptr(x, bf, "x"), _ptr(router_w, _f32(), "router_w"),
            _ptr(router_bias, _f32(), "router_bias", True), _ptr(w_gate, bf, "w_gate"),
            _ptr(w_up, bf, "w_up"), _ptr(w_down, bf, "w_down"),
            _ptr(ws_gate, bf, "ws_gate", True), _ptr(ws_up, bf, "ws_up", True),
            _ptr(ws_down, bf, "ws_down", True), _ptr(y, bf, "y"),
            _ptr(topk_ids_out, _i32(), "topk_ids_out", True),
            _ptr(topk_w_out, _f32(), "topk_w_out", True)]
    if not no_ws:
        args += [_ptr(ws, None, "ws"), ws.numel() * ws.element_size()]
    return args + [_stream(stream)]


def moe_forward(cfg, x, router_w, router_bias, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, y,
                topk_ids_out=None, topk_w_out=None, ws=None, stream=None):
    lib = load_library()
    _check(lib.moe_forward(*_forward_args(cfg, x, router_w, router_bias, w_gate, w_up, w_down,
                                          ws_gate, ws_up, ws_down, y, topk_ids_out, topk_w_out,
                                          ws, stream)))


def moe_forward_fused(cfg, x, router_w, router_bias, w_gate, w_up, w_down, ws_gate, ws_up,
                      ws_down, y, topk_ids_out=None, topk_w_out=None, ws=None, stream=None):
    """moe_forward in a single launch (tokens <= 256, tokens * top_k <= 2048)."""
    lib = load_library()
    _check(lib.moe_forward_fused(*_forward_args(cfg, x, router_w, router_bias, w_gate, w_up,
                                                w_down, ws_gate, ws_up, ws_down, y, topk_ids_out,
                                                topk_w_out, ws, stream)))


def moe_forward_noalloc(cfg, x, router_w, router_bias, w_gate, w_up, w_down, ws_gate, ws_up,
                        ws_down, y, topk_ids_out=None, topk_w_out=None, stream=None):
    """moe_forward with the library's fixed scratch as its workspace (no
    workspace argument, nothing allocated)."""
    lib = load_library()
    args = _forward_args(cfg, x, router_w, router_bias, w_gate, w_up, w_down, ws_gate, ws_up,
                         ws_down, y, topk_ids_out, topk_w_out, None, stream, no_ws=True)
    _check(lib.moe_forward_noalloc(*args))


def moe_forward_timed(cfg, x, router_w, router_bias, w_gate, w_up, w_down, ws_gate, ws_up,
                      ws_down, y, topk_ids_out=None, topk_w_out=None, ws=None, stream=None,
                      events=None):
    """`events`: MOE_NUM_STAGES + 1 torch.cuda.Event(enable_timing=True)."""
    lib = load_library()
    if events is None or len(events) != MOE_NUM_STAGES + 1:
        raise ValueError(f"need {MOE_NUM_STAGES + 1} events")
    handles = []
    for ev in events:
        if ev.cuda_event == 0:  # torch creates the HIP event lazily
            ev.record(_torch().cuda.current_stream())
        handles.append(ev.cuda_event)
    arr = (ctypes.c_void_p * len(handles))(*handles)
    _check(lib.moe_forward_timed(*_forward_args(cfg, x, router_w, router_bias, w_gate, w_up,
                                                w_down, ws_gate, ws_up, ws_down, y, topk_ids_out,
                                                topk_w_out, ws, stream), arr, len(handles)))


def moe_workspace_view(cfg, which: int):
    """(byte offset, byte size) of an intermediate inside the workspace."""
    lib = load_library()
    off, nb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib.moe_workspace_view(ctypes.byref(cfg), int(which), ctypes.byref(off),
                                  ctypes.byref(nb)))
    return int(off.value), int(nb.value)


# --------------------------------------------------------- layer wrapper

@dataclasses.dataclass
class MoeWeights:
    """Device tensors of one MoE layer (bf16 tensors may be torch.bfloat16 or
    raw-bit uint16/int16)."""
    router_w: object
    router_b: object
    w_gate: object
    w_up: object
    w_down: object
    ws_gate: object = None
    ws_up: object = None
    ws_down: object = None


def forward(cfg: moe_config, x, weights: MoeWeights, y=None, ws=None, topk_ids=None,
            topk_w=None, stream=None):
    """Allocate what is missing (output, workspace) and run moe_forward."""
    torch = _torch()
    if y is None:
        y = torch.empty((cfg.tokens, cfg.hidden), dtype=torch.bfloat16, device=x.device)
    if ws is None:
        ws = alloc_workspace(cfg, x.device)
    sh = cfg.inter_shared > 0
    moe_forward(cfg, x, weights.router_w, weights.router_b, weights.w_gate, weights.w_up,
                weights.w_down, weights.ws_gate if sh else None, weights.ws_up if sh else None,
                weights.ws_down if sh else None, y, topk_ids, topk_w, ws, stream)
    return y


# ------------------------------------------------------------------ dense FFN

def moe_dense_workspace_size(cfg: moe_dense_config) -> int:
    n = load_library().moe_dense_workspace_size(ctypes.byref(cfg))
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, moe_last_error())
    return int(n)


def alloc_dense_workspace(cfg: moe_dense_config, device=None):
    torch = _torch()
    return torch.empty(moe_dense_workspace_size(cfg), dtype=torch.uint8,
                       device=device or torch.device("cuda"))


def moe_dense_forward(cfg, x, w_gate, w_up, w_down, y, ws, stream=None):
    lib = load_library()
    _check(lib.moe_dense_forward(ctypes.byref(cfg), _ptr(x, _bf16(), "x", cfg.tokens == 0),
                                 _ptr(w_gate, _bf16(), "w_gate"), _ptr(w_up, _bf16(), "w_up"),
                                 _ptr(w_down, _bf16(), "w_down"),
                                 _ptr(y, _bf16(), "y", cfg.tokens == 0),
                                 _ptr(ws, None, "ws"), ws.numel() * ws.element_size(),
                                 _stream(stream)))


# ------------------------------------------------------------------ FP8 experts

def _u8():
    return (_torch().uint8, _torch().float8_e4m3fn)


def moe_forward_fp8(cfg, x, router_w, router_bias, w8_gate, w8_up, w8_down, scale_gate, scale_up,
                    scale_down, ws_gate, ws_up, ws_down, y, topk_ids_out, topk_w_out, ws,
                    stream=None):
    lib = load_library()
    empty = cfg.tokens == 0
    _check(lib.moe_forward_fp8(
        ctypes.byref(cfg), _ptr(x, _bf16(), "x", empty), _ptr(router_w, _f32(), "router_w"),
        _ptr(router_bias, _f32(), "router_bias", True), _ptr(w8_gate, _u8(), "w8_gate"),
        _ptr(w8_up, _u8(), "w8_up"), _ptr(w8_down, _u8(), "w8_down"),
        _ptr(scale_gate, _f32(), "scale_gate"), _ptr(scale_up, _f32(), "scale_up"),
        _ptr(scale_down, _f32(), "scale_down"), _ptr(ws_gate, _bf16(), "ws_gate", True),
        _ptr(ws_up, _bf16(), "ws_up", True), _ptr(ws_down, _bf16(), "ws_down", True),
        _ptr(y, _bf16(), "y", empty), _ptr(topk_ids_out, _i32(), "topk_ids_out", True),
        _ptr(topk_w_out, _f32(), "topk_w_out", True), _ptr(ws, None, "ws"),
        ws.numel() * ws.element_size(), _stream(stream)))


# ------------------------------------------------------------------ linear and grouped products

class _Args:
    """Checks of one call's tensors, in the order cheapest for tensors that
    pass (a call of a few microseconds of GPU work spends as long here
    otherwise), and the errors for those that do not."""
    __slots__ = ("device",)
    torch = None  # with the types below, set at the first call

    def __init__(self):
        if _Args.torch is None:
            torch = _torch()
            _Args.bf16 = (torch.bfloat16, torch.uint16, torch.int16)
            _Args.f32, _Args.i32 = (torch.float32,), (torch.int32,)
            _Args.u8 = (torch.uint8, torch.float8_e4m3fn)
            _Args.Tensor = torch.Tensor
            _Args.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            # (current_device by itself checks the initialisation again: 0.1 us)
            _Args.raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
            _Args.torch = torch
        # -2: no tensor's device (a host tensor's is -1)
        self.device = _Args.raw_device() if self.torch.cuda.is_initialized() else -2

    def __call__(self, t, name, dtypes, shape, optional=False):
        """Device address of a contiguous tensor on the current device: of
        `shape`, or the same memory in other dimensions, of which the last
        ones together make up a row (heads of a row, batches of rows), or
        flat."""
        if t is None and optional:
            return None
        try:
            if (t.dtype in dtypes and t.shape == shape and t.is_contiguous()
                    and t.get_device() == self.device):
                return t.data_ptr()
        except AttributeError:  # not a tensor
            pass
        _ptr(t, dtypes, name)
        numel, row = math.prod(shape), shape[-1]
        if t.numel() != numel:
            raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
        if t.dim() > 1 and row not in itertools.accumulate(reversed(t.shape), operator.mul):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected rows of {row}")
        return self._elsewhere(t, name)

    def rows(self, t, name, cfg):
        """Device address of a bf16 [rows][inter] tensor or view with the
        configuration's row stride."""
        ld = cfg.ld or cfg.inter
        if (isinstance(t, self.Tensor) and t.dtype in self.bf16
                and t.get_device() == self.device and t.shape == (cfg.rows, cfg.inter)
                and (t.stride() == (ld, 1) or cfg.rows == 1 and t.stride(1) == 1)):
            return t.data_ptr()
        if not isinstance(t, self.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be on the GPU, got {t.device}")
        if t.dtype not in self.bf16:
            raise TypeError(f"{name} has dtype {t.dtype}, expected one of {self.bf16}")
        if t.shape != (cfg.rows, cfg.inter):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(cfg.rows, cfg.inter)}")
        if t.stride(1) != 1 or (cfg.rows > 1 and t.stride(0) != ld):
            raise ValueError(f"{name} has strides {t.stride()}, expected ({ld}, 1)")
        return self._elsewhere(t, name)

    def of(self, dtype):
        """Tensor types of a MOE_DTYPE_*."""
        return self.f32 if dtype == 1 else self.bf16

    def workspace(self, ws):
        """(address, bytes) of a workspace tensor."""
        if ws is None:
            raise ValueError("ws is required")
        if (isinstance(ws, self.Tensor) and ws.is_contiguous()
                and ws.get_device() == self.device):
            return ws.data_ptr(), ws.nbytes
        p = _ptr(ws, None, "ws")
        self._elsewhere(ws, "ws")
        return p, ws.nbytes

    def stream(self, stream):
        """The HIP stream: `stream`, or torch's current one (by its raw handle
        where torch gives it: a Stream object costs 2.5 us)."""
        if stream is None and self.raw_stream is not None and self.device >= 0:
            return _Args.raw_stream(self.device)
        return _stream(stream)

    def _elsewhere(self, t, name):
        if t.get_device() != self.device:
            raise ValueError(f"{name} is on {t.device}, the current device is "
                             f"cuda:{self.device}")
        return t.data_ptr()


def _alloc(nbytes, device):
    torch = _torch()
    return torch.empty(nbytes, dtype=torch.uint8, device=device or torch.device("cuda"))


def moe_linear_workspace_size(cfg: moe_linear_config) -> int:
    n = load_library().moe_linear_workspace_size(ctypes.byref(cfg))
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, moe_last_error())
    return int(n)


def alloc_linear_workspace(cfg: moe_linear_config, device=None):
    return _alloc(moe_linear_workspace_size(cfg), device)


def moe_linear_forward(cfg, x, w, bias, residual, y, z=None, ws=None, stream=None):
    """z = x W^T + bias; y = act(z) + residual (bias, residual, z: may be None)."""
    T, K, F = cfg.tokens, cfg.in_features, cfg.out_features
    a = _Args()
    bf = a.bf16
    _check(load_library().moe_linear_forward(
        ctypes.byref(cfg), a(x, "x", bf, (T, K)), a(w, "w", bf, (F, K)),
        a(bias, "bias", a.f32, (F,), True), a(residual, "residual", bf, (T, F), True),
        a(y, "y", a.of(cfg.y_dtype), (T, F)), a(z, "z", bf, (T, F), True),
        *a.workspace(ws), a.stream(stream)))


def moe_linear_backward(cfg, dy, z, x, w, dz, dx, dw, dbias, ws=None, stream=None):
    """dz, dx, dw and dbias of moe_linear_forward for dy; dx, dw and dbias may
    be None, z and dz with activation "none"."""
    T, K, F = cfg.tokens, cfg.in_features, cfg.out_features
    a = _Args()
    bf = a.bf16
    plain = cfg.activation == 0
    _check(load_library().moe_linear_backward(
        ctypes.byref(cfg), a(dy, "dy", bf, (T, F)), a(z, "z", bf, (T, F), plain),
        a(x, "x", bf, (T, K), dw is None), a(w, "w", bf, (F, K), dx is None),
        a(dz, "dz", bf, (T, F), plain), a(dx, "dx", bf, (T, K), True),
        a(dw, "dw", a.of(cfg.dw_dtype), (F, K), True), a(dbias, "dbias", a.f32, (F,), True),
        *a.workspace(ws), a.stream(stream)))


def moe_grouped_workspace_size(cfg: moe_grouped_config) -> int:
    n = load_library().moe_grouped_workspace_size(ctypes.byref(cfg))
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, moe_last_error())
    return int(n)


def alloc_grouped_workspace(cfg: moe_grouped_config, device=None):
    return _alloc(moe_grouped_workspace_size(cfg), device)


def moe_grouped_forward(cfg, x, row_ids, offsets, w, bias, y, ws=None, stream=None):
    """y[r] = W_e x[src(r)] + bias_e for the rows r of each group e (row_ids
    and bias: may be None)."""
    P, E, K, F = cfg.rows, cfg.num_groups, cfg.in_features, cfg.out_features
    a = _Args()
    bf = a.bf16
    _check(load_library().moe_grouped_forward(
        ctypes.byref(cfg), a(x, "x", bf, (cfg.x_rows, K)),
        a(row_ids, "row_ids", a.i32, (P,), True), a(offsets, "offsets", a.i32, (E + 1,)),
        a(w, "w", bf, (E, F, K)), a(bias, "bias", a.f32, (E, F), True),
        a(y, "y", a.of(cfg.y_dtype), (P, F)),
        *a.workspace(ws), a.stream(stream)))


def moe_grouped_backward(cfg, dy, x, row_ids, offsets, w, dx, dw, dbias, ws=None, stream=None):
    """dx, dw and dbias of moe_grouped_forward for dy (each may be None)."""
    P, E, K, F = cfg.rows, cfg.num_groups, cfg.in_features, cfg.out_features
    a = _Args()
    bf = a.bf16
    _check(load_library().moe_grouped_backward(
        ctypes.byref(cfg), a(dy, "dy", bf, (P, F)), a(x, "x", bf, (cfg.x_rows, K), dw is None),
        a(row_ids, "row_ids", a.i32, (P,), True), a(offsets, "offsets", a.i32, (E + 1,)),
        a(w, "w", bf, (E, F, K), dx is None), a(dx, "dx", bf, (P, K), True),
        a(dw, "dw", a.of(cfg.dw_dtype), (E, F, K), True),
        a(dbias, "dbias", a.f32, (E, F), True),
        *a.workspace(ws), a.stream(stream)))


def moe_swiglu_forward(cfg, gate, up, h, stream=None):
    """h = SiLU(min(gate, L)) * clamp(up, -L, L); gate and up may be the halves
    of one [rows][2 inter] tensor (ld = 2 inter)."""
    a = _Args()
    _check(load_library().moe_swiglu_forward(
        ctypes.byref(cfg), a.rows(gate, "gate", cfg), a.rows(up, "up", cfg),
        a(h, "h", a.bf16, (cfg.rows, cfg.inter)), a.stream(stream)))


def moe_swiglu_backward(cfg, dh, gate, up, dgate, dup, h=None, stream=None):
    """dgate and dup for dh; h (may be None) is recomputed on the way."""
    n = (cfg.rows, cfg.inter)
    a = _Args()
    _check(load_library().moe_swiglu_backward(
        ctypes.byref(cfg), a(dh, "dh", a.bf16, n), a.rows(gate, "gate", cfg),
        a.rows(up, "up", cfg), a.rows(dgate, "dgate", cfg), a.rows(dup, "dup", cfg),
        a(h, "h", a.bf16, n, True), a.stream(stream)))


# ------------------------------------------------------------------ rows out to the experts and back

def moe_dispatch_forward(cfg, x, pair_pos, rows, stream=None):
    """rows[pair_pos[t][j]] = x[t] for every pair whose position is a row."""
    T, R, k, H = cfg.tokens, cfg.rows, cfg.top_k, cfg.hidden
    a = _Args()
    _check(load_library().moe_dispatch_forward(
        ctypes.byref(cfg), a(x, "x", a.of(cfg.token_dtype), (T, H)),
        a(pair_pos, "pair_pos", a.i32, (T, k)), a(rows, "rows", a.of(cfg.row_dtype), (R, H)),
        a.stream(stream)))


def moe_dispatch_backward(cfg, drows, pair_pos, base, dx, stream=None):
    """dx[t] = base[t] + sum_j drows[pair_pos[t][j]] (base: may be None)."""
    T, R, k, H = cfg.tokens, cfg.rows, cfg.top_k, cfg.hidden
    a = _Args()
    tok = a.of(cfg.token_dtype)
    _check(load_library().moe_dispatch_backward(
        ctypes.byref(cfg), a(drows, "drows", a.of(cfg.row_dtype), (R, H)),
        a(pair_pos, "pair_pos", a.i32, (T, k)), a(base, "base", tok, (T, H), True),
        a(dx, "dx", tok, (T, H)), a.stream(stream)))


def moe_combine_forward(cfg, rows, pair_pos, weights, base, y, stream=None):
    """y[t] = base[t] + sum_j weights[t][j] rows[pair_pos[t][j]] (weights, for
    ones, and base: may be None)."""
    T, R, k, H = cfg.tokens, cfg.rows, cfg.top_k, cfg.hidden
    a = _Args()
    tok = a.of(cfg.token_dtype)
    _check(load_library().moe_combine_forward(
        ctypes.byref(cfg), a(rows, "rows", a.of(cfg.row_dtype), (R, H)),
        a(pair_pos, "pair_pos", a.i32, (T, k)), a(weights, "weights", a.f32, (T, k), True),
        a(base, "base", tok, (T, H), True), a(y, "y", tok, (T, H)), a.stream(stream)))


def moe_combine_backward(cfg, dy, rows, pair_pos, weights, drows, dweights, stream=None):
    """drows[pair_pos[t][j]] = weights[t][j] dy[t] and dweights[t][j] = <dy[t],
    rows[pair_pos[t][j]]> (each may be None; rows without dweights)."""
    T, R, k, H = cfg.tokens, cfg.rows, cfg.top_k, cfg.hidden
    a = _Args()
    row = a.of(cfg.row_dtype)
    _check(load_library().moe_combine_backward(
        ctypes.byref(cfg), a(dy, "dy", a.of(cfg.token_dtype), (T, H)),
        a(rows, "rows", row, (R, H), dweights is None), a(pair_pos, "pair_pos", a.i32, (T, k)),
        a(weights, "weights", a.f32, (T, k), True), a(drows, "drows", row, (R, H), True),
        a(dweights, "dweights", a.f32, (T, k), True), a.stream(stream)))


# ------------------------------------------------------------------ products in 8 bits

def _blocks(n):
    return (n + 127) // 128


def moe_quantize_rows(cfg, x, pair_pos, codes, scales, stream=None):
    """e4m3 codes and scales (a block of 128 columns each) of x's rows; with
    pair_pos (else None), at the rows that it names."""
    T, R, k, K = cfg.tokens, cfg.rows, cfg.top_k, cfg.features
    a = _Args()
    _check(load_library().moe_quantize_rows(
        ctypes.byref(cfg), a(x, "x", a.bf16, (T, K)), a(pair_pos, "pair_pos", a.i32, (T, k), True),
        a(codes, "codes", a.u8, (R, K)), a(scales, "scales", a.f32, (R, _blocks(K))),
        a.stream(stream)))


def moe_quantize_weight(w, codes, scales, stream=None):
    """e4m3 codes and scales (a block of 128 x 128 each) of weights [F][K] or
    [G][F][K]."""
    a = _Args()
    if not isinstance(w, a.Tensor) or w.dim() not in (2, 3):
        raise ValueError("w must be a tensor of [F][K] or [G][F][K]")
    F, K = w.shape[-2:]
    G = w.shape[0] if w.dim() == 3 else 1
    _check(load_library().moe_quantize_weight(
        G, F, K, a(w, "w", a.bf16, tuple(w.shape)), a(codes, "codes", a.u8, tuple(w.shape)),
        a(scales, "scales", a.f32, (G, _blocks(F), _blocks(K))), a.stream(stream)))


def moe_linear_fp8_workspace_size(cfg: moe_linear_config) -> int:
    n = load_library().moe_linear_fp8_workspace_size(ctypes.byref(cfg))
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, moe_last_error())
    return int(n)


def alloc_linear_fp8_workspace(cfg: moe_linear_config, device=None):
    return _alloc(moe_linear_fp8_workspace_size(cfg), device)


def moe_linear_forward_fp8(cfg, x, x_scales, w, w_scales, bias, residual, y, z=None, ws=None,
                           stream=None):
    """moe_linear_forward of codes x and w with their scales."""
    T, K, F = cfg.tokens, cfg.in_features, cfg.out_features
    a = _Args()
    _check(load_library().moe_linear_forward_fp8(
        ctypes.byref(cfg), a(x, "x", a.u8, (T, K)), a(x_scales, "x_scales", a.f32, (T, _blocks(K))),
        a(w, "w", a.u8, (F, K)), a(w_scales, "w_scales", a.f32, (_blocks(F), _blocks(K))),
        a(bias, "bias", a.f32, (F,), True), a(residual, "residual", a.bf16, (T, F), True),
        a(y, "y", a.of(cfg.y_dtype), (T, F)), a(z, "z", a.bf16, (T, F), True),
        *a.workspace(ws), a.stream(stream)))


def moe_grouped_fp8_workspace_size(cfg: moe_grouped_config) -> int:
    n = load_library().moe_grouped_fp8_workspace_size(ctypes.byref(cfg))
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, moe_last_error())
    return int(n)


def alloc_grouped_fp8_workspace(cfg: moe_grouped_config, device=None):
    return _alloc(moe_grouped_fp8_workspace_size(cfg), device)


def moe_grouped_forward_fp8(cfg, x, x_scales, row_ids, offsets, w, w_scales, bias, y, ws=None,
                            stream=None):
    """moe_grouped_forward of codes x and w with their scales."""
    P, E, K, F = cfg.rows, cfg.num_groups, cfg.in_features, cfg.out_features
    a = _Args()
    _check(load_library().moe_grouped_forward_fp8(
        ctypes.byref(cfg), a(x, "x", a.u8, (cfg.x_rows, K)),
        a(x_scales, "x_scales", a.f32, (cfg.x_rows, _blocks(K))),
        a(row_ids, "row_ids", a.i32, (P,), True), a(offsets, "offsets", a.i32, (E + 1,)),
        a(w, "w", a.u8, (E, F, K)),
        a(w_scales, "w_scales", a.f32, (E, _blocks(F), _blocks(K))),
        a(bias, "bias", a.f32, (E, F), True), a(y, "y", a.of(cfg.y_dtype), (P, F)),
        *a.workspace(ws), a.stream(stream)))
