"""Thin ctypes binding of libbeam_moe.so (the C ABI in include/beam_moe.h).

Argument marshalling only: torch tensors supply device pointers and the
current HIP stream; every step of the block runs in the library's kernels.
The library is loaded from this package directory and nothing else: when it
is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

from .synth import Dims

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbeam_moe.so")

BEAM_MOE_OK = 0
BEAM_MOE_ERR_INVALID_ARG = -1
BEAM_MOE_ERR_UNSUPPORTED = -2
BEAM_MOE_ERR_WORKSPACE = -3
BEAM_MOE_ERR_HIP = -4
BEAM_MOE_ERR_SCRATCH = -5
SCRATCH_BYTES = 64 << 20       # BEAM_MOE_SCRATCH_BYTES: scratch of beam_moe_forward_noalloc

EXPORTED = ("beam_moe_workspace_bytes", "beam_moe_route_workspace_bytes", "beam_moe_dispatch_workspace_bytes",
            "beam_moe_route", "beam_moe_select", "beam_moe_dispatch",
            "beam_moe_forward", "beam_moe_forward_noalloc", "beam_moe_pack_weights", "beam_moe_forward_packed",
            "beam_moe_forward_fp8", "beam_moe_residual_forward",
            "beam_moe_residual_forward_fp8", "beam_moe_layer_norm", "beam_moe_layer_norm_backward_workspace_bytes",
            "beam_moe_layer_norm_backward", "beam_moe_balance_loss_workspace_bytes", "beam_moe_balance_loss",
            "beam_moe_route_backward", "beam_moe_linear_workspace_bytes", "beam_moe_linear_backward_workspace_bytes",
            "beam_moe_linear", "beam_moe_linear_backward", "beam_moe_stream_rows", "beam_moe_timing_enable",
            "beam_moe_timing_read", "beam_moe_stage_name", "beam_moe_status_str")

SIZE_MAX = 2 ** 64 - 1

BEAM_MOE_BF16, BEAM_MOE_F16, BEAM_MOE_F32 = 0, 1, 2
ELEM_TYPES = {torch.bfloat16: BEAM_MOE_BF16, torch.float16: BEAM_MOE_F16, torch.float32: BEAM_MOE_F32}
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}


class BeamMoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: status {status} ({status_text(status)})")


class CDims(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("intermediate", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("num_groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("routed_scaling", ctypes.c_float)]


_lib: Optional[ctypes.CDLL] = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the built library (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m grouped_top_routing_fp32_amd.build`")
    lib = ctypes.CDLL(path)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    pd = ctypes.POINTER(CDims)
    for fn in ("beam_moe_workspace_bytes", "beam_moe_route_workspace_bytes", "beam_moe_dispatch_workspace_bytes"):
        getattr(lib, fn).argtypes = [pd, i32]
        getattr(lib, fn).restype = sz
    lib.beam_moe_status_str.argtypes = [ctypes.c_int]
    lib.beam_moe_status_str.restype = ctypes.c_char_p
    lib.beam_moe_route.argtypes = [pd, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.beam_moe_route.restype = ctypes.c_int
    lib.beam_moe_select.argtypes = [pd, i32, vp, vp, vp, vp, vp]
    lib.beam_moe_select.restype = ctypes.c_int
    lib.beam_moe_dispatch.argtypes = [pd, i32, vp, vp, vp, vp, vp, sz, vp]
    lib.beam_moe_dispatch.restype = ctypes.c_int
    lib.beam_moe_forward.argtypes = [pd, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.beam_moe_forward.restype = ctypes.c_int
    lib.beam_moe_pack_weights.argtypes = [pd, vp, vp, vp]
    lib.beam_moe_pack_weights.restype = ctypes.c_int
    lib.beam_moe_forward_packed.argtypes = [pd, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.beam_moe_forward_packed.restype = ctypes.c_int
    lib.beam_moe_forward_noalloc.argtypes = [pd, i32] + [vp] * 13 + [vp]
    lib.beam_moe_forward_noalloc.restype = ctypes.c_int
    lib.beam_moe_forward_fp8.argtypes = [pd, i32] + [vp] * 17 + [sz, vp]
    lib.beam_moe_forward_fp8.restype = ctypes.c_int
    lib.beam_moe_residual_forward.argtypes = [pd, i32, vp, i32, vp, vp, ctypes.c_float, vp, vp, vp, vp, vp, vp, vp,
                                              vp, vp, vp, vp, vp, vp, sz, vp]
    lib.beam_moe_residual_forward.restype = ctypes.c_int
    lib.beam_moe_residual_forward_fp8.argtypes = [pd, i32, vp, i32, vp, vp, ctypes.c_float] + [vp] * 16 + [sz, vp]
    lib.beam_moe_residual_forward_fp8.restype = ctypes.c_int
    ci, i64, f32 = ctypes.c_int, ctypes.c_int64, ctypes.c_float
    for fn, res, args in (
            ("beam_moe_layer_norm", ci, [i32, i32, vp, ci, i64, vp, vp, f32, vp, ci, i64, vp, vp, vp]),
            ("beam_moe_layer_norm_backward_workspace_bytes", sz, [i32, i32]),
            ("beam_moe_layer_norm_backward", ci,
             [i32, i32, vp, ci, i64, vp, ci, i64, vp, vp, vp, vp, i64, vp, vp, vp, sz, vp]),
            ("beam_moe_balance_loss_workspace_bytes", sz, [pd, i32, i32]),
            ("beam_moe_balance_loss", ci, [pd, i32, vp, vp, i32, vp, f32, vp, vp, vp, vp, sz, vp]),
            ("beam_moe_route_backward", ci, [pd, i32, vp, vp, vp, i32, vp, f32, vp, vp, vp, vp]),
            ("beam_moe_linear_workspace_bytes", sz, [i32, i32, i32, i64, i64]),
            ("beam_moe_linear_backward_workspace_bytes", sz, [i32, i32, i32, i64, i64]),
            ("beam_moe_linear", ci, [i32, i32, i32, ci, vp, i64, vp, i64, vp, ci, vp, i64, f32, f32, vp, ci, i64, vp,
                                     i64, vp, sz, vp]),
            ("beam_moe_linear_backward", ci, [i32, i32, i32, ci, vp, ci, i64, vp, i64, vp, i64, vp, i64, ci, f32, f32,
                                              vp, i64, vp, i64, vp, vp, i64, vp, sz, vp])):
        getattr(lib, fn).argtypes = args
        getattr(lib, fn).restype = res
    lib.beam_moe_stream_rows.argtypes = [pd, i32, ctypes.c_int]
    lib.beam_moe_stream_rows.restype = ctypes.c_int
    lib.beam_moe_timing_enable.argtypes = [ctypes.c_int]
    lib.beam_moe_timing_enable.restype = ctypes.c_int
    lib.beam_moe_timing_read.argtypes = [ctypes.POINTER(ctypes.c_float), i32, ctypes.POINTER(i32),
                                         ctypes.POINTER(i32)]
    lib.beam_moe_timing_read.restype = ctypes.c_int
    lib.beam_moe_stage_name.argtypes = [i32]
    lib.beam_moe_stage_name.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_text(status: int) -> str:
    try:
        return load_library().beam_moe_status_str(status).decode()
    except Exception:  # the message of an error must not itself raise
        return "?"


def _cdims(d: Dims) -> CDims:
    return CDims(d.hidden, d.intermediate, d.num_experts, d.num_groups, d.topk_groups, d.topk,
                 float(d.routed_scaling))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(status: int, what: str) -> None:
    if status != BEAM_MOE_OK:
        raise BeamMoeError(status, what)


def _req(t: torch.Tensor, name: str, dtype: torch.dtype, shape) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# --------------------------------------------------------------------------
# raw entry points (same names as the C ABI)
# --------------------------------------------------------------------------
def _ws_query(fn: str, dims: Dims, T: int) -> int:
    cd = _cdims(dims)
    n = getattr(load_library(), fn)(ctypes.byref(cd), int(T))
    if n == SIZE_MAX:
        raise BeamMoeError(BEAM_MOE_ERR_UNSUPPORTED, fn)
    return int(n)


def beam_moe_workspace_bytes(dims: Dims, T: int) -> int:
    return _ws_query("beam_moe_workspace_bytes", dims, T)


def beam_moe_route_workspace_bytes(dims: Dims, T: int) -> int:
    return _ws_query("beam_moe_route_workspace_bytes", dims, T)


def beam_moe_dispatch_workspace_bytes(dims: Dims, T: int) -> int:
    return _ws_query("beam_moe_dispatch_workspace_bytes", dims, T)


def beam_moe_status_str(status: int) -> str:
    return status_text(status)


def workspace(dims: Dims, T: int, device="cuda", size_fn=None) -> torch.Tensor:
    """A uint8 device buffer of size_fn(dims, T) bytes (default beam_moe_workspace_bytes)."""
    n = (size_fn or beam_moe_workspace_bytes)(dims, T)
    return torch.empty(max(16, n), dtype=torch.uint8, device=device)


def beam_moe_route(dims: Dims, x: torch.Tensor, w_router: torch.Tensor, logit_bias: Optional[torch.Tensor] = None,
                   *, select_bias: Optional[torch.Tensor] = None, want_scores: bool = False,
                   ws: Optional[torch.Tensor] = None, stream=None):
    """Router + group-limited top-k. Returns (ids [T,K] int32, w [T,K] f32, scores [T,E] f32 or None)."""
    T = x.shape[0]
    H, E, K = dims.hidden, dims.num_experts, dims.topk
    _req(x, "x", torch.bfloat16, (T, H))
    _req(w_router, "w_router", torch.float32, (E, H))
    if logit_bias is not None:
        _req(logit_bias, "logit_bias", torch.float32, (E,))
    if select_bias is not None:
        _req(select_bias, "select_bias", torch.float32, (E,))
    dev = x.device
    ids = torch.empty((T, K), dtype=torch.int32, device=dev)
    w = torch.empty((T, K), dtype=torch.float32, device=dev)
    scores = torch.empty((T, E), dtype=torch.float32, device=dev) if want_scores else None
    if ws is None:
        ws = workspace(dims, T, dev, beam_moe_route_workspace_bytes)
    cd = _cdims(dims)
    st = load_library().beam_moe_route(ctypes.byref(cd), T, _ptr(x), _ptr(w_router), _ptr(logit_bias),
                                       _ptr(select_bias), _ptr(ids), _ptr(w), _ptr(scores), _ptr(ws), ws.numel(),
                                       _stream(stream))
    _check(st, "beam_moe_route")
    return ids, w, scores


def beam_moe_select(dims: Dims, scores: torch.Tensor, *, select_bias: Optional[torch.Tensor] = None, stream=None):
    """Selection on supplied post-sigmoid FP32 scores [T,E]. Returns (ids, w)."""
    T = scores.shape[0]
    _req(scores, "scores", torch.float32, (T, dims.num_experts))
    if select_bias is not None:
        _req(select_bias, "select_bias", torch.float32, (dims.num_experts,))
    ids = torch.empty((T, dims.topk), dtype=torch.int32, device=scores.device)
    w = torch.empty((T, dims.topk), dtype=torch.float32, device=scores.device)
    cd = _cdims(dims)
    st = load_library().beam_moe_select(ctypes.byref(cd), T, _ptr(scores), _ptr(select_bias), _ptr(ids), _ptr(w),
                                        _stream(stream))
    _check(st, "beam_moe_select")
    return ids, w


def beam_moe_dispatch(dims: Dims, topk_ids: torch.Tensor, *, ws: Optional[torch.Tensor] = None, stream=None):
    """Counting-sort dispatch. Returns (counts [E], offsets [E+1], sorted_slots [T*K]) int32."""
    T = topk_ids.shape[0]
    _req(topk_ids, "topk_ids", torch.int32, (T, dims.topk))
    dev = topk_ids.device
    E = dims.num_experts
    counts = torch.empty((E,), dtype=torch.int32, device=dev)
    offsets = torch.empty((E + 1,), dtype=torch.int32, device=dev)
    slots = torch.empty((T * dims.topk,), dtype=torch.int32, device=dev)
    if ws is None:
        ws = workspace(dims, T, dev, beam_moe_dispatch_workspace_bytes)
    cd = _cdims(dims)
    st = load_library().beam_moe_dispatch(ctypes.byref(cd), T, _ptr(topk_ids), _ptr(counts), _ptr(offsets),
                                          _ptr(slots), _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "beam_moe_dispatch")
    return counts, offsets, slots


class ForwardBuffers:
    """Caller-owned outputs and workspace of beam_moe_forward for T tokens."""

    def __init__(self, dims: Dims, T: int, device="cuda"):
        E, K, H = dims.num_experts, dims.topk, dims.hidden
        self.T = T
        self.out = torch.empty((T, H), dtype=torch.float32, device=device)
        self.ids = torch.empty((T, K), dtype=torch.int32, device=device)
        self.w = torch.empty((T, K), dtype=torch.float32, device=device)
        self.counts = torch.empty((E,), dtype=torch.int32, device=device)
        self.offsets = torch.empty((E + 1,), dtype=torch.int32, device=device)
        self.slots = torch.empty((T * K,), dtype=torch.int32, device=device)
        self.ws = workspace(dims, T, device)


def _req_router(dims: Dims, w_router, logit_bias, select_bias) -> None:
    E, H = dims.num_experts, dims.hidden
    _req(w_router, "w_router", torch.float32, (E, H))
    for t, name in ((logit_bias, "logit_bias"), (select_bias, "select_bias")):
        if t is not None:
            _req(t, name, torch.float32, (E,))


def _req_bf16_experts(dims: Dims, w_gate, w_up, w_down) -> None:
    E, I, H = dims.num_experts, dims.intermediate, dims.hidden
    _req(w_gate, "w_gate", torch.bfloat16, (E, I, H))
    _req(w_up, "w_up", torch.bfloat16, (E, I, H))
    _req(w_down, "w_down", torch.bfloat16, (E, H, I))


def _req_fp8_experts(dims: Dims, w_gate_fp8, gate_scale, w_up_fp8, up_scale, w_down_fp8, down_scale) -> None:
    E, I, H = dims.num_experts, dims.intermediate, dims.hidden
    _req(w_gate_fp8, "w_gate_fp8", torch.uint8, (E, I, H))
    _req(w_up_fp8, "w_up_fp8", torch.uint8, (E, I, H))
    _req(w_down_fp8, "w_down_fp8", torch.uint8, (E, H, I))
    _req(gate_scale, "gate_scale", torch.float32, (E, I))
    _req(up_scale, "up_scale", torch.float32, (E, I))
    _req(down_scale, "down_scale", torch.float32, (E, H))


def _buffers(dims: Dims, T: int, device, bufs: Optional[ForwardBuffers]) -> ForwardBuffers:
    if bufs is None:
        return ForwardBuffers(dims, T, device)
    if bufs.T != T:
        raise ValueError("buffers were sized for another T")
    return bufs


def _outputs(bufs: ForwardBuffers, out: torch.Tensor):
    """Pointer arguments from `out` through the workspace, as every forward entry point takes them."""
    return (_ptr(out), _ptr(bufs.ids), _ptr(bufs.w), _ptr(bufs.counts), _ptr(bufs.offsets), _ptr(bufs.slots),
            _ptr(bufs.ws), bufs.ws.numel())


def beam_moe_forward(dims: Dims, x: torch.Tensor, w_router: torch.Tensor, logit_bias: Optional[torch.Tensor],
                     w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, *,
                     select_bias: Optional[torch.Tensor] = None, bufs: Optional[ForwardBuffers] = None,
                     stream=None) -> ForwardBuffers:
    """The whole block. Returns the ForwardBuffers holding out and the routing by-products."""
    T = x.shape[0]
    _req(x, "x", torch.bfloat16, (T, dims.hidden))
    _req_router(dims, w_router, logit_bias, select_bias)
    _req_bf16_experts(dims, w_gate, w_up, w_down)
    bufs = _buffers(dims, T, x.device, bufs)
    cd = _cdims(dims)
    st = load_library().beam_moe_forward(
        ctypes.byref(cd), T, _ptr(x), _ptr(w_router), _ptr(logit_bias), _ptr(select_bias), _ptr(w_gate), _ptr(w_up),
        _ptr(w_down), *_outputs(bufs, bufs.out), _stream(stream))
    _check(st, "beam_moe_forward")
    return bufs


def beam_moe_pack_weights(dims: Dims, w_down: torch.Tensor, out: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """W_down [E, H, I] bf16 -> fp16 (the form beam_moe_forward_packed takes)."""
    E, I, H = dims.num_experts, dims.intermediate, dims.hidden
    _req(w_down, "w_down", torch.bfloat16, (E, H, I))
    if out is None:
        out = torch.empty((E, H, I), dtype=torch.float16, device=w_down.device)
    _req(out, "w_down_packed", torch.float16, (E, H, I))
    cd = _cdims(dims)
    _check(load_library().beam_moe_pack_weights(ctypes.byref(cd), _ptr(w_down), _ptr(out), _stream(stream)),
           "beam_moe_pack_weights")
    return out


def beam_moe_forward_packed(dims: Dims, x: torch.Tensor, w_router: torch.Tensor,
                            logit_bias: Optional[torch.Tensor], w_gate: torch.Tensor, w_up: torch.Tensor,
                            w_down_packed: torch.Tensor, *, select_bias: Optional[torch.Tensor] = None,
                            bufs: Optional[ForwardBuffers] = None, stream=None) -> ForwardBuffers:
    """beam_moe_forward with W_down from beam_moe_pack_weights (fp16)."""
    T = x.shape[0]
    E, I, H = dims.num_experts, dims.intermediate, dims.hidden
    _req(x, "x", torch.bfloat16, (T, H))
    _req_router(dims, w_router, logit_bias, select_bias)
    _req(w_gate, "w_gate", torch.bfloat16, (E, I, H))
    _req(w_up, "w_up", torch.bfloat16, (E, I, H))
    _req(w_down_packed, "w_down_packed", torch.float16, (E, H, I))
    bufs = _buffers(dims, T, x.device, bufs)
    cd = _cdims(dims)
    st = load_library().beam_moe_forward_packed(
        ctypes.byref(cd), T, _ptr(x), _ptr(w_router), _ptr(logit_bias), _ptr(select_bias), _ptr(w_gate), _ptr(w_up),
        _ptr(w_down_packed), *_outputs(bufs, bufs.out), _stream(stream))
    _check(st, "beam_moe_forward_packed")
    return bufs


def beam_moe_forward_noalloc(dims: Dims, x: torch.Tensor, w_router: torch.Tensor,
                             logit_bias: Optional[torch.Tensor], w_gate: torch.Tensor, w_up: torch.Tensor,
                             w_down: torch.Tensor, *, select_bias: Optional[torch.Tensor] = None,
                             bufs: Optional[ForwardBuffers] = None, stream=None) -> ForwardBuffers:
    """beam_moe_forward on the library's built-in scratch (no workspace); bufs.ws is not used."""
    T = x.shape[0]
    _req(x, "x", torch.bfloat16, (T, dims.hidden))
    _req_router(dims, w_router, logit_bias, select_bias)
    _req_bf16_experts(dims, w_gate, w_up, w_down)
    bufs = _buffers(dims, T, x.device, bufs)
    cd = _cdims(dims)
    st = load_library().beam_moe_forward_noalloc(
        ctypes.byref(cd), T, _ptr(x), _ptr(w_router), _ptr(logit_bias), _ptr(select_bias), _ptr(w_gate), _ptr(w_up),
        _ptr(w_down), *_outputs(bufs, bufs.out)[:6], _stream(stream))
    _check(st, "beam_moe_forward_noalloc")
    return bufs


def beam_moe_forward_fp8(dims: Dims, x: torch.Tensor, w_router: torch.Tensor, logit_bias: Optional[torch.Tensor],
                         w_gate_fp8: torch.Tensor, gate_scale: torch.Tensor, w_up_fp8: torch.Tensor,
                         up_scale: torch.Tensor, w_down_fp8: torch.Tensor, down_scale: torch.Tensor, *,
                         select_bias: Optional[torch.Tensor] = None, bufs: Optional[ForwardBuffers] = None,
                         stream=None) -> ForwardBuffers:
    """The whole block with E4M3 expert weights (uint8 codes) and fp32 per-row scales."""
    T = x.shape[0]
    _req(x, "x", torch.bfloat16, (T, dims.hidden))
    _req_router(dims, w_router, logit_bias, select_bias)
    _req_fp8_experts(dims, w_gate_fp8, gate_scale, w_up_fp8, up_scale, w_down_fp8, down_scale)
    bufs = _buffers(dims, T, x.device, bufs)
    cd = _cdims(dims)
    st = load_library().beam_moe_forward_fp8(
        ctypes.byref(cd), T, _ptr(x), _ptr(w_router), _ptr(logit_bias), _ptr(select_bias), _ptr(w_gate_fp8),
        _ptr(gate_scale), _ptr(w_up_fp8), _ptr(up_scale), _ptr(w_down_fp8), _ptr(down_scale),
        *_outputs(bufs, bufs.out), _stream(stream))
    _check(st, "beam_moe_forward_fp8")
    return bufs


def _residual_prelude(dims: Dims, stream_in, norm_in_weight, norm_out_weight, stream_out, bufs):
    T = stream_in.shape[0]
    H = dims.hidden
    _req(stream_in, "stream_in", torch.float32, (T, H))
    for t, name in ((norm_in_weight, "norm_in_weight"), (norm_out_weight, "norm_out_weight")):
        if t is not None:
            _req(t, name, torch.float32, (H,))
    bufs = _buffers(dims, T, stream_in.device, bufs)
    if stream_out is not None:
        _req(stream_out, "stream_out", torch.float32, (T, H))
    return T, bufs, (stream_out if stream_out is not None else bufs.out)


def beam_moe_residual_forward(dims: Dims, stream_in: torch.Tensor, step: int, w_router: torch.Tensor,
                              logit_bias: Optional[torch.Tensor], w_gate: torch.Tensor, w_up: torch.Tensor,
                              w_down: torch.Tensor, *, select_bias: Optional[torch.Tensor] = None,
                              norm_in_weight: Optional[torch.Tensor] = None,
                              norm_out_weight: Optional[torch.Tensor] = None, norm_eps: float = 1e-6,
                              stream_out: Optional[torch.Tensor] = None, bufs: Optional[ForwardBuffers] = None,
                              stream=None) -> ForwardBuffers:
    """The block as a residual sublayer at `step`: the new stream goes to stream_out if given (it may be
    stream_in itself), else to bufs.out; the routing by-products to bufs."""
    T, bufs, out = _residual_prelude(dims, stream_in, norm_in_weight, norm_out_weight, stream_out, bufs)
    _req_router(dims, w_router, logit_bias, select_bias)
    _req_bf16_experts(dims, w_gate, w_up, w_down)
    cd = _cdims(dims)
    st = load_library().beam_moe_residual_forward(
        ctypes.byref(cd), T, _ptr(stream_in), int(step), _ptr(norm_in_weight), _ptr(norm_out_weight),
        float(norm_eps), _ptr(w_router), _ptr(logit_bias), _ptr(select_bias), _ptr(w_gate), _ptr(w_up),
        _ptr(w_down), *_outputs(bufs, out), _stream(stream))
    _check(st, "beam_moe_residual_forward")
    return bufs


def beam_moe_residual_forward_fp8(dims: Dims, stream_in: torch.Tensor, step: int, w_router: torch.Tensor,
                                  logit_bias: Optional[torch.Tensor], w_gate_fp8: torch.Tensor,
                                  gate_scale: torch.Tensor, w_up_fp8: torch.Tensor, up_scale: torch.Tensor,
                                  w_down_fp8: torch.Tensor, down_scale: torch.Tensor, *,
                                  select_bias: Optional[torch.Tensor] = None,
                                  norm_in_weight: Optional[torch.Tensor] = None,
                                  norm_out_weight: Optional[torch.Tensor] = None, norm_eps: float = 1e-6,
                                  stream_out: Optional[torch.Tensor] = None, bufs: Optional[ForwardBuffers] = None,
                                  stream=None) -> ForwardBuffers:
    """beam_moe_residual_forward with E4M3 expert weights and fp32 per-row scales."""
    T, bufs, out = _residual_prelude(dims, stream_in, norm_in_weight, norm_out_weight, stream_out, bufs)
    _req_router(dims, w_router, logit_bias, select_bias)
    _req_fp8_experts(dims, w_gate_fp8, gate_scale, w_up_fp8, up_scale, w_down_fp8, down_scale)
    cd = _cdims(dims)
    st = load_library().beam_moe_residual_forward_fp8(
        ctypes.byref(cd), T, _ptr(stream_in), int(step), _ptr(norm_in_weight), _ptr(norm_out_weight),
        float(norm_eps), _ptr(w_router), _ptr(logit_bias), _ptr(select_bias), _ptr(w_gate_fp8), _ptr(gate_scale),
        _ptr(w_up_fp8), _ptr(up_scale), _ptr(w_down_fp8), _ptr(down_scale), *_outputs(bufs, out), _stream(stream))
    _check(st, "beam_moe_residual_forward_fp8")
    return bufs


# --------------------------------------------------------------------------
# operators around the block: layer norm, the router's training side, linear
# --------------------------------------------------------------------------
# the current stream's handle without a Stream object around it, which takes 2.7 us to make
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class _On:
    """Where a call runs: the tensors' device made current, and the given stream, or that device's
    current one.  Outputs and workspaces allocated inside belong to that stream."""
    __slots__ = ("dev", "stream", "ctx")

    def __init__(self, dev: torch.device, stream):
        self.dev, self.stream, self.ctx = dev, stream, None

    def __enter__(self) -> int:
        dev, stream = self.dev, self.stream
        if stream is None:
            if torch.cuda.current_device() != dev.index:
                self.ctx = torch.cuda.device(dev)
                self.ctx.__enter__()
            return _raw_stream(dev.index)
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=dev)
        elif stream.device != dev:
            raise ValueError(f"the stream belongs to {stream.device}, the tensors to {dev}")
        self.ctx = torch.cuda.stream(stream)
        self.ctx.__enter__()
        return stream.cuda_stream

    def __exit__(self, *exc) -> None:
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _rows(t: torch.Tensor, name: str, dtypes, shape: tuple, dev) -> int:
    """Checks a matrix whose rows may be strided; returns its row stride."""
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, as the first tensor is")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {tuple(dtypes)}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    r, c = shape
    ld, one = t.stride()
    if one != 1 and c > 1:
        raise ValueError(f"{name} must have consecutive columns")
    if ld >= c:
        return ld
    if r > 1:
        raise ValueError(f"{name} must have rows that do not overlap")
    return c


def _vec(t: Optional[torch.Tensor], name: str, dtype, shape, dev) -> Optional[int]:
    """Checks an optional contiguous tensor; returns its address."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {dev}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _mat(t: torch.Tensor, name: str) -> tuple:
    """Rows, columns and device of the matrix that the others are checked against."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return *t.shape, t.device


def _result(out: Optional[torch.Tensor], out_dtype, default, dtypes, shape: tuple, dev):
    """The output and its row stride: the caller's, checked, or a new one."""
    if out is None:
        dtype = out_dtype or default
        if dtype not in dtypes:
            raise ValueError(f"out_dtype must be one of {tuple(dtypes)}, got {dtype}")
        return torch.empty(*shape, dtype=dtype, device=dev), shape[1]
    if out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out is not of out_dtype")
    return out, _rows(out, "out", dtypes, shape, dev)


def _scratch(n: int, ws: Optional[torch.Tensor], dev, fn: str):
    """(address, bytes, keeper) of a workspace of n bytes: the caller's, or a new one."""
    if n == SIZE_MAX:
        raise BeamMoeError(BEAM_MOE_ERR_UNSUPPORTED, fn)
    if ws is None:
        if n == 0:
            return None, 0, None
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
    elif ws.device != dev or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous on {dev}")
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


_cdims_of = functools.lru_cache(maxsize=64)(_cdims)


@functools.lru_cache(maxsize=4096)
def _linear_ws(fn: str, *sizes: int) -> int:
    """A workspace query of sizes alone, remembered: the call through ctypes takes 0.6 us, a tenth of a small
    product's time on the host."""
    return getattr(load_library(), fn)(*sizes)


_FLOATS = tuple(ELEM_TYPES)
_F32 = torch.float32


def beam_moe_layer_norm(x: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None, *,
                        eps: float = 1e-5, out_dtype: Optional[torch.dtype] = None,
                        out: Optional[torch.Tensor] = None, want_stats: bool = True, stream=None):
    """Layer norm of the rows of x [T, H] (bf16, fp16 or fp32; rows may be strided). Returns (y, mean, rstd):
    y of out_dtype (default x's), mean and rstd [T] fp32 for the backward pass, or None without want_stats."""
    T, H, dev = _mat(x, "x")
    ldx = _rows(x, "x", _FLOATS, (T, H), dev)
    g, b = _vec(gamma, "gamma", _F32, (H,), dev), _vec(beta, "beta", _F32, (H,), dev)
    with _On(dev, stream) as st:
        out, ldy = _result(out, out_dtype, x.dtype, _FLOATS, (T, H), dev)
        mean = torch.empty(T, dtype=_F32, device=dev) if want_stats else None
        rstd = torch.empty_like(mean) if want_stats else None
        _check(load_library().beam_moe_layer_norm(
            T, H, x.data_ptr(), ELEM_TYPES[x.dtype], ldx, g, b, eps, out.data_ptr(), ELEM_TYPES[out.dtype], ldy,
            mean.data_ptr() if want_stats else None, rstd.data_ptr() if want_stats else None, st),
            "beam_moe_layer_norm")
    return out, mean, rstd


def beam_moe_layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                                 gamma: Optional[torch.Tensor] = None, *, want_dx: bool = True,
                                 want_params: bool = True, ws: Optional[torch.Tensor] = None, stream=None):
    """Gradients of beam_moe_layer_norm. Returns (dx of x's type, dgamma [H] fp32, dbeta [H] fp32); dx is None
    without want_dx, the other two without want_params."""
    T, H, dev = _mat(x, "x")
    ldx, lddy = _rows(x, "x", _FLOATS, (T, H), dev), _rows(dy, "dy", _FLOATS, (T, H), dev)
    m, r = _vec(mean, "mean", _F32, (T,), dev), _vec(rstd, "rstd", _F32, (T,), dev)
    g = _vec(gamma, "gamma", _F32, (H,), dev)
    lib = load_library()
    with _On(dev, stream) as st:
        dx = torch.empty(T, H, dtype=x.dtype, device=dev) if want_dx else None
        dg = torch.empty(H, dtype=_F32, device=dev) if want_params else None
        db = torch.empty_like(dg) if want_params else None
        need = lib.beam_moe_layer_norm_backward_workspace_bytes(T, H) if want_params else 0
        wp, wn, _keep = _scratch(need, ws, dev, "beam_moe_layer_norm_backward")
        _check(lib.beam_moe_layer_norm_backward(
            T, H, dy.data_ptr(), ELEM_TYPES[dy.dtype], lddy, x.data_ptr(), ELEM_TYPES[x.dtype], ldx, m, r, g,
            dx.data_ptr() if want_dx else None, H, dg.data_ptr() if want_params else None,
            db.data_ptr() if want_params else None, wp, wn, st), "beam_moe_layer_norm_backward")
    return dx, dg, db


def _routed(dims: Dims, scores: torch.Tensor, topk_ids: torch.Tensor, seq_offsets: Optional[torch.Tensor]):
    T, E, dev = _mat(scores, "scores")
    s = _vec(scores, "scores", _F32, (T, dims.num_experts), dev)
    i = _vec(topk_ids, "topk_ids", torch.int32, (T, dims.topk), dev)
    B = 1
    if seq_offsets is not None:
        B = seq_offsets.numel() - 1
        if B < 1:
            raise ValueError("seq_offsets must hold at least two offsets")
    return T, E, dev, s, i, B, _vec(seq_offsets, "seq_offsets", torch.int32, (B + 1,), dev)


def beam_moe_balance_loss(dims: Dims, scores: torch.Tensor, topk_ids: torch.Tensor, *, alpha: float,
                          seq_offsets: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """Load-balance loss and per-expert counts of each packed sequence (one sequence without seq_offsets
    [B+1] int32). Returns (loss [B] fp32, counts [B,E] int32, prob [B,E] fp32)."""
    T, E, dev, s, i, B, off = _routed(dims, scores, topk_ids, seq_offsets)
    lib, cd = load_library(), _cdims_of(dims)
    with _On(dev, stream) as st:
        loss = torch.empty(B, dtype=_F32, device=dev)
        prob = torch.empty(B, E, dtype=_F32, device=dev)
        counts = torch.empty_like(prob, dtype=torch.int32)
        wp, wn, _keep = _scratch(lib.beam_moe_balance_loss_workspace_bytes(ctypes.byref(cd), T, B), ws, dev,
                                 "beam_moe_balance_loss")
        _check(lib.beam_moe_balance_loss(ctypes.byref(cd), T, s, i, B, off, alpha, loss.data_ptr(), counts.data_ptr(),
                                         prob.data_ptr(), wp, wn, st), "beam_moe_balance_loss")
    return loss, counts, prob


def beam_moe_route_backward(dims: Dims, scores: torch.Tensor, topk_ids: torch.Tensor, *,
                            dw: Optional[torch.Tensor] = None, dloss: Optional[torch.Tensor] = None,
                            counts: Optional[torch.Tensor] = None, alpha: float = 0.0,
                            seq_offsets: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient with respect to the router's logits, [T,E] fp32, of the routing weights (given dw [T,K]) and of
    beam_moe_balance_loss (given dloss [B] and its counts, alpha and seq_offsets)."""
    T, E, dev, s, i, B, off = _routed(dims, scores, topk_ids, seq_offsets)
    d = _vec(dw, "dw", _F32, (T, dims.topk), dev)
    dl, c = _vec(dloss, "dloss", _F32, (B,), dev), _vec(counts, "counts", torch.int32, (B, E), dev)
    cd = _cdims_of(dims)
    with _On(dev, stream) as st:
        out = torch.empty_like(scores)
        if T == 0 and (dw is not None or dloss is not None):
            return out
        _check(load_library().beam_moe_route_backward(ctypes.byref(cd), T, s, i, d, B, off, alpha, dl, c,
                                                      out.data_ptr(), st), "beam_moe_route_backward")
    return out


_HALF = (torch.bfloat16, torch.float16)


def _act(act: str) -> int:
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {tuple(ACTIVATIONS)}, got {act!r}")
    return ACTIVATIONS[act]


def beam_moe_linear(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, *, act: str = "none",
                    residual: Optional[torch.Tensor] = None, keep: float = 1.0, add: float = 1.0,
                    out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                    want_pre: bool = False, ws: Optional[torch.Tensor] = None, stream=None):
    """y = keep * residual + add * act(x w^T + bias) for x [M, K], w [N, K] in bf16 or fp16 (rows may be strided),
    bias [N] fp32. y is of out_dtype (x's type, or fp32), as residual is; out may be residual itself. Returns y,
    or (y, pre) with want_pre: pre [M, N] of x's type is what the backward pass reads."""
    M, K, dev = _mat(x, "x")
    if w.dim() != 2:
        raise ValueError("w must be a matrix")
    N = w.shape[0]
    ldx, ldw = _rows(x, "x", _HALF, (M, K), dev), _rows(w, "w", (x.dtype,), (N, K), dev)
    b, a = _vec(bias, "bias", _F32, (N,), dev), _act(act)
    lib = load_library()
    with _On(dev, stream) as st:
        out, ldy = _result(out, out_dtype, x.dtype, (x.dtype, _F32), (M, N), dev)
        ldr = 0 if residual is None else _rows(residual, "residual", (out.dtype,), (M, N), dev)
        pre = torch.empty(M, N, dtype=x.dtype, device=dev) if want_pre else None
        wp, wn, _keep = _scratch(_linear_ws("beam_moe_linear_workspace_bytes", M, N, K, ldx, ldw), ws, dev,
                                 "beam_moe_linear")
        _check(lib.beam_moe_linear(
            M, N, K, ELEM_TYPES[x.dtype], x.data_ptr(), ldx, w.data_ptr(), ldw, b, a,
            None if residual is None else residual.data_ptr(), ldr, keep, add, out.data_ptr(), ELEM_TYPES[out.dtype],
            ldy, pre.data_ptr() if want_pre else None, N, wp, wn, st), "beam_moe_linear")
    return (out, pre) if want_pre else out


def beam_moe_linear_backward(dy: torch.Tensor, x: Optional[torch.Tensor], w: Optional[torch.Tensor],
                             pre: Optional[torch.Tensor] = None, *, act: str = "none", keep: float = 1.0,
                             add: float = 1.0, want_dx: bool = True, want_dw: bool = True, want_dbias: bool = True,
                             want_dres: bool = False, ws: Optional[torch.Tensor] = None, stream=None):
    """Gradients of beam_moe_linear from dy [M, N] (x's type or fp32) and, with an activation, pre. Returns
    (dx, dw, dbias), with want_dres (dx, dw, dbias, dres); those not wanted are None. x may be None without
    want_dw, w without want_dx; one of them is needed for the type."""
    if x is None and w is None or want_dw and x is None or want_dx and w is None:
        raise ValueError("x is needed for dw, w for dx, and one of them for the type")
    M, N, dev = _mat(dy, "dy")
    K, dt = (x if x is not None else w).shape[-1], (x if x is not None else w).dtype
    if dt not in _HALF:
        raise ValueError(f"x and w must be one of {_HALF}, got {dt}")
    ldx = K if x is None else _rows(x, "x", _HALF, (M, K), dev)
    ldw = K if w is None else _rows(w, "w", (dt,), (N, K), dev)
    lddy = _rows(dy, "dy", (dt, _F32), (M, N), dev)
    a = _act(act)
    ldp = N
    if a:
        if pre is None:
            raise ValueError("pre is needed with an activation")
        ldp = _rows(pre, "pre", (dt,), (M, N), dev)
    lib = load_library()
    with _On(dev, stream) as st:
        dx = torch.empty(M, K, dtype=dt, device=dev) if want_dx else None
        dw = torch.empty(N, K, dtype=dt, device=dev) if want_dw else None
        db = torch.empty(N, dtype=_F32, device=dev) if want_dbias else None
        dres = torch.empty(M, N, dtype=dy.dtype, device=dev) if want_dres else None
        wp, wn, _keep = _scratch(_linear_ws("beam_moe_linear_backward_workspace_bytes", M, N, K, ldx, ldw), ws, dev,
                                 "beam_moe_linear_backward")
        _check(lib.beam_moe_linear_backward(
            M, N, K, ELEM_TYPES[dt], dy.data_ptr(), ELEM_TYPES[dy.dtype], lddy, None if x is None else x.data_ptr(),
            ldx, None if w is None else w.data_ptr(), ldw, pre.data_ptr() if a else None, ldp, a, keep, add,
            dx.data_ptr() if want_dx else None, K, dw.data_ptr() if want_dw else None, K,
            db.data_ptr() if want_dbias else None, dres.data_ptr() if want_dres else None, N, wp, wn, st),
            "beam_moe_linear_backward")
    return (dx, dw, db, dres) if want_dres else (dx, dw, db)


# --------------------------------------------------------------------------
# stage timing diagnostics
# --------------------------------------------------------------------------
def beam_moe_stream_rows(dims: Dims, T: int, fp8: bool = False) -> int:
    """Rows per stream-kernel tile the forward entry points use for T tokens, or 0 for the grouped GEMMs."""
    cd = _cdims(dims)
    r = load_library().beam_moe_stream_rows(ctypes.byref(cd), int(T), int(bool(fp8)))
    if r < 0:
        raise BeamMoeError(r, "beam_moe_stream_rows")
    return r


def beam_moe_timing_enable(enable: bool = True) -> None:
    _check(load_library().beam_moe_timing_enable(int(bool(enable))), "beam_moe_timing_enable")


def beam_moe_stage_name(stage: int) -> Optional[str]:
    r = load_library().beam_moe_stage_name(stage)
    return None if r is None else r.decode()


def beam_moe_timing_read() -> tuple[dict, int]:
    """({stage name: summed ms}, calls) since the previous read; waits for the last recorded call."""
    buf = (ctypes.c_float * 16)()
    ns, calls = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(load_library().beam_moe_timing_read(buf, 16, ctypes.byref(ns), ctypes.byref(calls)),
           "beam_moe_timing_read")
    return {beam_moe_stage_name(i): float(buf[i]) for i in range(ns.value)}, calls.value
