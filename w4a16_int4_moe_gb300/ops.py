"""Thin ctypes binding of ``libw4a16moe.so`` (declared in include/w4a16moe.h).

Names follow the C entry points. Every function only marshals arguments:
tensors become ``data_ptr()`` values, the stream is torch's current CUDA
stream. All computation happens in the library's CUDA kernels; a missing or
unloadable library raises ``RuntimeError`` (there is no CPU fallback).
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

from . import build as _build

W4A16_OK = 0
W4A16_ERR_INVALID_ARG = 1
W4A16_ERR_UNSUPPORTED = 2
W4A16_ERR_ROUTING = 3
W4A16_ERR_WORKSPACE = 4
W4A16_ERR_CUDA = 5
W4A16_ERR_TIMEOUT = 6

W4A16_GATE_UP = 0
W4A16_DOWN = 1
W4A16_GATE_UP_SILU = 2
W4A16_GROUPED_CONTIGUOUS = 0
W4A16_GROUPED_MASKED = 1
W4A16_FLAG_VALIDATE_ROUTING = 1
W4A16_FLAG_ACCUMULATE = 2
W4A16_FLAG_DETERMINISTIC = 8
W4A16_LAYOUT_KTILE64 = 0
W4A16_LAYOUT_KTILE64_GLU16 = 1
W4A16_DTYPE_F32 = 0
W4A16_DTYPE_BF16 = 1
W4A16_DTYPE_FP8 = 2
W4A16_FP8_NONE = 0
W4A16_FP8_ROW = -1
W4A16_FP8_GROUP = 128
W4A16_FEW_TOKENS_MAX = 32
W4A16_FLAG_SYNC_STATUS = 4

# Every symbol include/w4a16moe.h declares.
EXPORTED = (
    "w4a16_status_string", "w4a16_version", "w4a16_plan", "w4a16_align_capacity",
    "w4a16_moe_align_block_size", "w4a16_prepack_size", "w4a16_prepack", "w4a16_unpack",
    "w4a16_workspace_size", "w4a16_moe_indexed_gemm", "w4a16_moe_grouped_gemm",
    "w4a16_silu_and_mul", "w4a16_read_device_status", "w4a16_moe_indexed_gemm_noalloc",
    "w4a16_topk_softmax", "w4a16_deterministic_bytes", "w4a16_layer_workspace_size",
    "w4a16_moe_layer", "w4a16_moe_route_align", "w4a16_grouped_plan", "w4a16_plan_info",
    "w4a16_add_rms_norm", "w4a16_router_logits", "w4a16_moe_few_tokens_workspace_size",
    "w4a16_moe_few_tokens", "w4a16_linear_few_tokens", "w4a16_dense", "w4a16_block_norm",
    "w4a16_dense_info",
)


class Plan(ctypes.Structure):
    """Mirror of w4a16_plan_t."""
    _fields_ = [(name, ctypes.c_int) for name in (
        "block_m", "bn", "bk", "stages", "b_stages", "split_k", "ctas_per_sm", "swap_ab",
        "layout", "grid", "cta_pair")]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class PlanInfo(ctypes.Structure):
    """Mirror of w4a16_plan_info_t."""
    _fields_ = [(name, ctypes.c_int) for name in (
        "mma_issuers", "acc_slots", "acc_cols", "early_epilogue", "w_stages", "b_stages")] + [
        ("smem_bytes", ctypes.c_size_t)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class DenseInfo(ctypes.Structure):
    """w4a16_dense_info_t."""
    _fields_ = [(name, ctypes.c_int) for name in ("kernel", "tile_rows", "split", "run")]


class W4A16Error(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} failed: status {status} ({msg})")
        self.status = status


_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_Z = ctypes.c_size_t
_L = ctypes.c_longlong
_F = ctypes.c_float


def load_library(path: Optional[str] = None):
    """Load the library (building it first when it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    if path is None:
        path = _build.LIB
        if _build.is_stale():
            _build.build_library()
    if not os.path.exists(path):
        raise RuntimeError(f"W4A16 MoE CUDA library not found at {path}")
    lib = ctypes.CDLL(path)
    sig = {
        "w4a16_status_string": (ctypes.c_char_p, [_I]),
        "w4a16_version": (_I, []),
        "w4a16_plan": (_I, [_I, _I, _I, _I, _I, ctypes.c_float, ctypes.POINTER(Plan)]),
        "w4a16_align_capacity": (_Z, [_I, _I, _I]),
        "w4a16_grouped_plan": (_I, [_I, _I, _I, _I, _I, ctypes.POINTER(Plan)]),
        "w4a16_plan_info": (_I, [ctypes.POINTER(Plan), _I, ctypes.POINTER(PlanInfo)]),
        "w4a16_moe_align_block_size": (_I, [_P, _I, _I, _I, _I, _I, _P, _P, _P, _P]),
        "w4a16_prepack_size": (_I, [_I, _I, _I, _I, _I, ctypes.POINTER(_Z)]),
        "w4a16_prepack": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _Z, _P]),
        "w4a16_unpack": (_I, [_P, _I, _I, _I, _I, _P, _P, _P]),
        "w4a16_workspace_size": (_Z, [ctypes.POINTER(Plan), _I, _I]),
        "w4a16_deterministic_bytes": (_Z, [_I, _I, _I]),
        "w4a16_moe_indexed_gemm": (_I, [_I, _P, _I, _I, _I, _P, _I, _I, _P, _P, _P, _I, _P, _P,
                                        _I, ctypes.POINTER(Plan), _P, _Z, _P]),
        "w4a16_moe_grouped_gemm": (_I, [_I, _P, _I, _I, _I, _P, _I, _P, _I, _P, _I,
                                        ctypes.POINTER(Plan), _P, _Z, _P]),
        "w4a16_silu_and_mul": (_I, [_P, _I, _I, _P, _P]),
        "w4a16_topk_softmax": (_I, [_P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P]),
        "w4a16_moe_route_align": (_I, [_P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P,
                                       _P, _P, _P]),
        "w4a16_read_device_status": (_I, [_P, ctypes.POINTER(_I), _P]),
        "w4a16_layer_workspace_size": (_Z, [ctypes.POINTER(Plan), _I, _I, _I]),
        "w4a16_moe_layer": (_I, [_P, _P, _I, _I, _I, _P, _I, _I, _P, _P, _P, _I, _P, _P, _I,
                                 ctypes.POINTER(Plan), _P, _Z, _P]),
        "w4a16_moe_indexed_gemm_noalloc": (_I, [_I, _P, _I, _I, _I, _P, _I, _I, _P, _P, _P, _I,
                                                _P, _P, _I, ctypes.POINTER(Plan), _P]),
        "w4a16_add_rms_norm": (_I, [_P, _L, _P, _L, _P, _F, _I, _I, _P, _P, _P, _P, _I, _P]),
        "w4a16_router_logits": (_I, [_P, _L, _P, _I, _I, _I, _P, _P]),
        "w4a16_moe_few_tokens_workspace_size": (_Z, [_I, _I, _I, _I]),
        "w4a16_moe_few_tokens": (_I, [_P, _P, _I, _I, _I, _P, _I, _P, _I, _I, _P, _I, _I, _I, _I,
                                      _P, _P, _P, _I, _P, _Z, _P]),
        "w4a16_linear_few_tokens": (_I, [_P, _I, _I, _I, _P, _L, _I, _P, _P, _I, _P]),
        "w4a16_dense": (_I, [_P, _I, _I, _I, _P, _L, _I, _P, _P, _I, _P]),
        "w4a16_dense_info": (_I, [_I, _I, _I, _I, _I, _P, _P]),
        "w4a16_block_norm": (_I, [_P, _I, _L, _P, _P, _L, _P, _L, _P, _F, _F, _F, _F, _I, _I, _P,
                                  _P, _P, _P, _I, _P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().w4a16_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != W4A16_OK:
        raise W4A16Error(fn, status, status_string(status))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


_HERE = contextlib.nullcontext()


def on_stream(stream):
    """The context in which a call makes its memory: what is allocated (or
    filled, or copied) inside belongs to the stream that the call runs on, so
    that the allocator hands it on only behind that stream's work. None: the
    current stream, as without a context."""
    return _HERE if stream is None else torch.cuda.stream(stream)


# ------------------------------------------------------------- host only --

def w4a16_version() -> int:
    return load_library().w4a16_version()


def w4a16_plan(tokens: int, topk: int, num_experts: int, n: int, k: int,
               tok_e_hint: float = 0.0) -> Plan:
    p = Plan()
    _check("w4a16_plan", load_library().w4a16_plan(tokens, topk, num_experts, n, k,
                                                    float(tok_e_hint), ctypes.byref(p)))
    return p


def w4a16_align_capacity(numel: int, num_experts: int, block_m: int) -> int:
    return int(load_library().w4a16_align_capacity(numel, num_experts, block_m))


def w4a16_prepack_size(num_experts: int, n: int, k: int, group: int = 32,
                       layout: int = W4A16_LAYOUT_KTILE64) -> int:
    out = _Z(0)
    _check("w4a16_prepack_size", load_library().w4a16_prepack_size(
        num_experts, n, k, group, layout, ctypes.byref(out)))
    return int(out.value)


def w4a16_grouped_plan(kind: int, m: int, n: int, k: int, expected_m: int = 0) -> Plan:
    """The plan w4a16_moe_grouped_gemm uses when given none."""
    p = Plan()
    _check("w4a16_grouped_plan", load_library().w4a16_grouped_plan(
        kind, m, expected_m, n, k, ctypes.byref(p)))
    return p


def w4a16_plan_info(plan: Plan, k: int) -> PlanInfo:
    """What a plan becomes on the device for reduction length k."""
    info = PlanInfo()
    _check("w4a16_plan_info", load_library().w4a16_plan_info(ctypes.byref(plan), k,
                                                             ctypes.byref(info)))
    return info


def w4a16_workspace_size(plan: Plan, rows: int = 0, k: int = 0) -> int:
    """rows: routing capacity of an indexed GEMM (0 for grouped); k: the
    GEMM's reduction length."""
    return int(load_library().w4a16_workspace_size(ctypes.byref(plan), rows, k))


# ---------------------------------------------------------------- device --

def w4a16_moe_align_block_size(topk_ids: torch.Tensor, num_experts: int, block_m: int,
                               capacity: Optional[int] = None, out=None, stream=None):
    """Returns (sorted_ids, expert_ids, num_tokens_padded) int32 device tensors."""
    tokens, topk = topk_ids.shape
    numel = tokens * topk
    if capacity is None:
        capacity = w4a16_align_capacity(numel, num_experts, block_m)
    dev = topk_ids.device
    if out is None:
        with on_stream(stream):
            out = (torch.empty(capacity, dtype=torch.int32, device=dev),
                   torch.empty(capacity // block_m, dtype=torch.int32, device=dev),
                   torch.empty(1, dtype=torch.int32, device=dev))
    sorted_ids, expert_ids, ntp = out
    _check("w4a16_moe_align_block_size", load_library().w4a16_moe_align_block_size(
        _ptr(topk_ids), tokens, topk, num_experts, block_m, capacity,
        _ptr(sorted_ids), _ptr(expert_ids), _ptr(ntp), _stream(stream)))
    return sorted_ids, expert_ids, ntp


def w4a16_prepack(q: torch.Tensor, scales: torch.Tensor, group: int = 32,
                  layout: int = W4A16_LAYOUT_KTILE64, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """q uint8 [E, n, k/2], scales BF16 [E, n, k/32] -> packed uint8 blob."""
    e, n, kh = q.shape
    k = kh * 2
    size = w4a16_prepack_size(e, n, k, group, layout)
    if out is None:
        with on_stream(stream):
            out = torch.empty(size, dtype=torch.uint8, device=q.device)
    _check("w4a16_prepack", load_library().w4a16_prepack(
        _ptr(q), _ptr(scales), e, n, k, group, layout, _ptr(out), out.numel(), _stream(stream)))
    return out


def w4a16_unpack(packed: torch.Tensor, num_experts: int, n: int, k: int,
                 layout: int = W4A16_LAYOUT_KTILE64, stream=None):
    with on_stream(stream):
        q = torch.empty((num_experts, n, k // 2), dtype=torch.uint8, device=packed.device)
        s = torch.empty((num_experts, n, k // 32), dtype=torch.int16, device=packed.device)
    _check("w4a16_unpack", load_library().w4a16_unpack(
        _ptr(packed), num_experts, n, k, layout, _ptr(q), _ptr(s), _stream(stream)))
    return q, s


def w4a16_deterministic_bytes(capacity: int, n: int, numel: int) -> int:
    """Extra workspace of a W4A16_FLAG_DETERMINISTIC down call."""
    return int(load_library().w4a16_deterministic_bytes(capacity, n, numel))


def new_workspace(plan: Plan, device, rows: int = 0, k: int = 0, det_n: int = 0,
                  det_numel: int = 0) -> torch.Tensor:
    """det_n, det_numel: room for a deterministic down pass of width det_n
    over det_numel flattened rows (0: none)."""
    size = w4a16_workspace_size(plan, rows, k)
    if det_n > 0:
        size += w4a16_deterministic_bytes(rows, det_n, det_numel)
    return torch.zeros(size, dtype=torch.uint8, device=device)


def w4a16_moe_indexed_gemm(mode: int, packed: torch.Tensor, num_experts: int, n: int, k: int,
                           a: torch.Tensor, tokens: int, topk: int, sorted_ids: torch.Tensor,
                           expert_ids: torch.Tensor, num_tokens_padded: torch.Tensor,
                           plan: Plan, workspace: torch.Tensor,
                           topk_weights: Optional[torch.Tensor] = None,
                           out: Optional[torch.Tensor] = None, flags: int = 0, stream=None):
    """GATE_UP: out BF16 [tokens*topk, n]; GATE_UP_SILU: out BF16
    [tokens*topk, n/2]; DOWN: out FP32 [tokens, n]."""
    if out is None:
        with on_stream(stream):
            if mode == W4A16_GATE_UP:
                out = torch.empty((tokens * topk, n), dtype=torch.bfloat16, device=a.device)
            elif mode == W4A16_GATE_UP_SILU:
                out = torch.empty((tokens * topk, n // 2), dtype=torch.bfloat16, device=a.device)
            else:
                out = torch.empty((tokens, n), dtype=torch.float32, device=a.device)
    _check("w4a16_moe_indexed_gemm", load_library().w4a16_moe_indexed_gemm(
        mode, _ptr(packed), num_experts, n, k, _ptr(a), tokens, topk, _ptr(sorted_ids),
        _ptr(expert_ids), _ptr(num_tokens_padded), sorted_ids.numel(), _ptr(topk_weights),
        _ptr(out), flags, ctypes.byref(plan), _ptr(workspace), workspace.numel(),
        _stream(stream)))
    return out


def w4a16_moe_grouped_gemm(kind: int, packed: torch.Tensor, num_experts: int, n: int, k: int,
                           a: torch.Tensor, m: int, layout: torch.Tensor, workspace: torch.Tensor,
                           plan: Optional[Plan] = None, expected_m: int = 0,
                           out: Optional[torch.Tensor] = None, flags: int = 0, stream=None):
    """CONTIGUOUS: a [m, k] -> out [m, n]; MASKED: a [E, m, k] -> out [E, m, n] (BF16)."""
    if out is None:
        shape = (m, n) if kind == W4A16_GROUPED_CONTIGUOUS else (num_experts, m, n)
        with on_stream(stream):
            out = torch.empty(shape, dtype=torch.bfloat16, device=a.device)
    _check("w4a16_moe_grouped_gemm", load_library().w4a16_moe_grouped_gemm(
        kind, _ptr(packed), num_experts, n, k, _ptr(a), m, _ptr(layout), expected_m, _ptr(out),
        flags, None if plan is None else ctypes.byref(plan), _ptr(workspace), workspace.numel(),
        _stream(stream)))
    return out


def w4a16_layer_workspace_size(plan: Plan, rows: int, hidden: int, inter: int) -> int:
    return int(load_library().w4a16_layer_workspace_size(ctypes.byref(plan), rows, hidden, inter))


def w4a16_moe_layer(packed_gate_up: torch.Tensor, packed_down: torch.Tensor, num_experts: int,
                    hidden: int, inter: int, x: torch.Tensor, tokens: int, topk: int,
                    sorted_ids: torch.Tensor, expert_ids: torch.Tensor,
                    num_tokens_padded: torch.Tensor, plan: Plan, workspace: torch.Tensor,
                    topk_weights: torch.Tensor, out: Optional[torch.Tensor] = None,
                    flags: int = 0, stream=None):
    """The layer's gate_up (fused activation) and down in one launch:
    out FP32 [tokens, hidden]."""
    if out is None:
        with on_stream(stream):
            out = torch.empty((tokens, hidden), dtype=torch.float32, device=x.device)
    _check("w4a16_moe_layer", load_library().w4a16_moe_layer(
        _ptr(packed_gate_up), _ptr(packed_down), num_experts, hidden, inter, _ptr(x), tokens,
        topk, _ptr(sorted_ids), _ptr(expert_ids), _ptr(num_tokens_padded), sorted_ids.numel(),
        _ptr(topk_weights), _ptr(out), flags, ctypes.byref(plan), _ptr(workspace),
        workspace.numel(), _stream(stream)))
    return out


def w4a16_topk_softmax(logits: torch.Tensor, topk: int, renormalize: bool = True,
                       expert_offset: int = 0, num_local_experts: Optional[int] = None,
                       out=None, stream=None):
    """logits fp32/BF16 [T, E] -> (topk_ids int32 [T, topk] local or -1,
    topk_weights fp32 [T, topk])."""
    tokens, e = logits.shape
    if num_local_experts is None:
        num_local_experts = e
    dtype = {torch.float32: W4A16_DTYPE_F32, torch.bfloat16: W4A16_DTYPE_BF16}.get(logits.dtype)
    if dtype is None:
        raise W4A16Error("w4a16_topk_softmax", W4A16_ERR_INVALID_ARG,
                         f"logits of dtype {logits.dtype}")
    if not logits.is_contiguous():
        with on_stream(stream):
            logits = logits.contiguous()
    if out is None:
        with on_stream(stream):
            out = (torch.empty((tokens, topk), dtype=torch.int32, device=logits.device),
                   torch.empty((tokens, topk), dtype=torch.float32, device=logits.device))
    ids, w = out
    _check("w4a16_topk_softmax", load_library().w4a16_topk_softmax(
        _ptr(logits), dtype, tokens, e, topk, int(bool(renormalize)), expert_offset,
        num_local_experts, _ptr(ids), _ptr(w), _stream(stream)))
    return ids, w


def w4a16_moe_route_align(logits: torch.Tensor, topk: int, block_m: int,
                          arrivals: torch.Tensor, renormalize: bool = True,
                          expert_offset: int = 0, num_local_experts: Optional[int] = None,
                          capacity: Optional[int] = None, out=None, stream=None):
    """Top-k routing and moe_align_block_size in one launch. arrivals: int32
    [1] device, zero before the first call (each call leaves it zero).
    Returns (topk_ids, topk_weights, sorted_ids, expert_ids, num_tokens_padded)."""
    tokens, e = logits.shape
    if num_local_experts is None:
        num_local_experts = e
    dtype = {torch.float32: W4A16_DTYPE_F32, torch.bfloat16: W4A16_DTYPE_BF16}.get(logits.dtype)
    if dtype is None:
        raise W4A16Error("w4a16_moe_route_align", W4A16_ERR_INVALID_ARG,
                         f"logits of dtype {logits.dtype}")
    if capacity is None:
        capacity = w4a16_align_capacity(tokens * topk, num_local_experts, block_m)
    dev = logits.device
    if not logits.is_contiguous():
        with on_stream(stream):
            logits = logits.contiguous()
    if out is None:
        with on_stream(stream):
            out = (torch.empty((tokens, topk), dtype=torch.int32, device=dev),
                   torch.empty((tokens, topk), dtype=torch.float32, device=dev),
                   torch.empty(capacity, dtype=torch.int32, device=dev),
                   torch.empty(capacity // block_m, dtype=torch.int32, device=dev),
                   torch.empty(1, dtype=torch.int32, device=dev))
    ids, w, sorted_ids, expert_ids, ntp = out
    _check("w4a16_moe_route_align", load_library().w4a16_moe_route_align(
        _ptr(logits), dtype, tokens, e, topk, int(bool(renormalize)), expert_offset,
        num_local_experts, block_m, sorted_ids.numel(), _ptr(ids), _ptr(w), _ptr(sorted_ids),
        _ptr(expert_ids), _ptr(ntp), _ptr(arrivals), _stream(stream)))
    return ids, w, sorted_ids, expert_ids, ntp


def w4a16_silu_and_mul(x: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None):
    rows, two_i = x.shape
    inter = two_i // 2
    if out is None:
        with on_stream(stream):
            out = torch.empty((rows, inter), dtype=torch.bfloat16, device=x.device)
    _check("w4a16_silu_and_mul", load_library().w4a16_silu_and_mul(
        _ptr(x), rows, inter, _ptr(out), _stream(stream)))
    return out


# The calls of the layer's latency-bound path (one token up to a small batch)
# pass plain integers: no ctypes object is built per pointer, and the current
# stream is read without making a Stream object.

_BF16, _E4M3, _F32, _I32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.int32
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # (of CUDA builds)


def _raw_stream(t: torch.Tensor, stream):
    return _current_stream(t.get_device()) if stream is None else stream.cuda_stream


def _refuse(fn: str, why: str):
    raise W4A16Error(fn, W4A16_ERR_INVALID_ARG, why)


def _need(fn: str, what: str, t: torch.Tensor, dtype, shape):
    """The address of t, a contiguous GPU tensor of this type and shape (else
    W4A16_ERR_INVALID_ARG)."""
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _refuse(fn, f"{what}: {t.dtype} {tuple(t.shape)} on {t.device}, "
                    f"not contiguous {dtype} {tuple(shape)} on a GPU")
    return t.data_ptr()


def _blob(fn: str, what: str, t: torch.Tensor, size: int):
    """The address of t, at least `size` contiguous bytes (uint8) on a GPU."""
    if t.dtype is not torch.uint8 or not t.is_cuda or not t.is_contiguous() or t.numel() < size:
        _refuse(fn, f"{what}: {t.numel()} x {t.dtype} on {t.device}, not {size} bytes on a GPU")
    return t.data_ptr()


def _rows(fn: str, what: str, t: torch.Tensor):
    """t is BF16 [rows, columns] on a GPU with adjacent columns; returns
    (address, rows, columns, row stride)."""
    if t.dtype is not _BF16 or not t.is_cuda or t.dim() != 2:
        _refuse(fn, f"{what}: {t.dtype} {tuple(t.shape)} on {t.device}")
    rows, columns = t.shape
    if t.is_contiguous():
        return t.data_ptr(), rows, columns, columns
    pitch, step = t.stride()
    if step != 1 and columns > 1:
        _refuse(fn, f"{what}: strides {t.stride()}")
    return t.data_ptr(), rows, columns, pitch if rows > 1 else max(pitch, columns)


def w4a16_add_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                       residual: Optional[torch.Tensor] = None,
                       fp8_group: int = W4A16_FP8_NONE, bf16_out: bool = True, out=None,
                       stream=None):
    """h = x + residual, y = h * rsqrt(mean(h^2) + eps) * weight.
    Returns (bf16(y), bf16(h), e4m3(y * (1 / scale)), scale), each None when not
    asked for: bf16_out, residual, fp8_group (W4A16_FP8_GROUP: a scale per 128
    columns, W4A16_FP8_ROW: one per row). out: the four tensors to write, None
    for an absent one (it then decides which of y and its 8-bit form is
    written, and the second entry may be the residual itself). x and residual
    BF16 [T, H], rows may be strided."""
    fn = "w4a16_add_rms_norm"
    x_at, rows, hidden, x_stride = _rows(fn, "x", x)
    w_at = _need(fn, "weight", weight, _BF16, (hidden,))
    r_at, r_stride = None, 0
    if residual is not None:
        r_at, r_rows, r_cols, r_stride = _rows(fn, "residual", residual)
        if r_rows != rows or r_cols != hidden:
            _refuse(fn, f"residual {tuple(residual.shape)} for x {tuple(x.shape)}")
    shape, groups = (rows, hidden), (rows, 0)
    if fp8_group != W4A16_FP8_NONE:
        if fp8_group not in (W4A16_FP8_ROW, W4A16_FP8_GROUP):
            raise W4A16Error(fn, W4A16_ERR_UNSUPPORTED, f"fp8_group {fp8_group}")
        groups = (rows, 1 if fp8_group == W4A16_FP8_ROW else -(-hidden // W4A16_FP8_GROUP))
    if out is None:
        kinds = ((shape, _BF16, bf16_out), (shape, _BF16, residual is not None),
                 (shape, _E4M3, fp8_group), (groups, _F32, fp8_group))
        with on_stream(stream):
            out = tuple(torch.empty(size, dtype=dtype, device=x.device) if wanted else None
                        for size, dtype, wanted in kinds)
    y, res_out, y8, scales = out
    _check(fn, load_library().w4a16_add_rms_norm(
        x_at, x_stride, r_at, r_stride, w_at, eps, rows, hidden,
        None if y is None else _need(fn, "out", y, _BF16, shape),
        None if res_out is None else _need(fn, "residual_out", res_out, _BF16, shape),
        None if y8 is None else _need(fn, "out_fp8", y8, _E4M3, shape),
        None if scales is None else _need(fn, "scales", scales, _F32, groups),
        fp8_group, _raw_stream(x, stream)))
    return out


def w4a16_router_logits(x: torch.Tensor, weight: torch.Tensor,
                        out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x BF16 [T, H] (rows may be strided), weight BF16 [E, H] -> FP32 [T, E]."""
    fn = "w4a16_router_logits"
    x_at, tokens, hidden, x_stride = _rows(fn, "x", x)
    experts = weight.shape[0]
    w_at = _need(fn, "weight", weight, _BF16, (experts, hidden))
    if out is None:
        with on_stream(stream):
            out = torch.empty((tokens, experts), dtype=torch.float32, device=x.device)
    _check(fn, load_library().w4a16_router_logits(
        x_at, x_stride, w_at, tokens, hidden, experts,
        _need(fn, "out", out, _F32, (tokens, experts)), _raw_stream(x, stream)))
    return out


def w4a16_moe_few_tokens_workspace_size(tokens: int, topk: int, hidden: int, inter: int) -> int:
    return int(load_library().w4a16_moe_few_tokens_workspace_size(tokens, topk, hidden, inter))


def w4a16_moe_few_tokens(packed_gate_up: torch.Tensor, packed_down: torch.Tensor,
                         num_experts: int, hidden: int, inter: int, x: torch.Tensor,
                         topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                         workspace: torch.Tensor, x_scales: Optional[torch.Tensor] = None,
                         logits: Optional[torch.Tensor] = None, renormalize: bool = True,
                         expert_offset: int = 0, out: Optional[torch.Tensor] = None,
                         flags: int = 0, stream=None) -> torch.Tensor:
    """The whole layer for up to W4A16_FEW_TOKENS_MAX tokens: out FP32 [T, H].
    x BF16 [T, H], or e4m3 [T, H] with x_scales FP32 [T, ceil(H/128)]. Without
    logits, topk_ids and topk_weights [T, topk] are the routing; with logits
    (FP32 or BF16 [T, E_global]) they receive it."""
    fn = "w4a16_moe_few_tokens"
    tokens, topk = picks = topk_ids.shape
    fp8 = x_scales is not None
    x_at = _need(fn, "x", x, _E4M3 if fp8 else _BF16, (tokens, hidden))
    s_at = None
    if fp8:
        s_at = _need(fn, "x_scales", x_scales, torch.float32,
                     (tokens, -(-hidden // W4A16_FP8_GROUP)))
    lg_at, lg_type, experts = None, W4A16_DTYPE_F32, 0
    if logits is not None:
        dtype = logits.dtype
        if dtype is torch.bfloat16:
            lg_type = W4A16_DTYPE_BF16
        else:
            dtype = torch.float32
        experts = logits.shape[1]
        lg_at = _need(fn, "logits", logits, dtype, (tokens, experts))
    if out is None:
        with on_stream(stream):
            out = torch.empty((tokens, hidden), dtype=torch.float32, device=x.device)
    # 128-row tiles of 64-column steps, 4608 bytes each
    gate_up_size = num_experts * -(-2 * inter // 128) * -(-hidden // 64) * 4608
    down_size = num_experts * -(-hidden // 128) * -(-inter // 64) * 4608
    _check(fn, load_library().w4a16_moe_few_tokens(
        _blob(fn, "packed_gate_up", packed_gate_up, gate_up_size),
        _blob(fn, "packed_down", packed_down, down_size), num_experts, hidden, inter, x_at,
        W4A16_DTYPE_FP8 if fp8 else W4A16_DTYPE_BF16, s_at, tokens, topk, lg_at, lg_type, experts,
        1 if renormalize else 0, expert_offset,
        _need(fn, "topk_ids", topk_ids, _I32, picks),
        _need(fn, "topk_weights", topk_weights, _F32, picks),
        _need(fn, "out", out, _F32, (tokens, hidden)), flags,
        _blob(fn, "workspace", workspace, 0), workspace.numel(), _raw_stream(x, stream)))
    return out


# The calls below take all tensors on one device, which need not be the current
# one: the library launches on the current device, so it is made current.

_current_device = getattr(torch._C, "_cuda_getDevice", None)  # (of CUDA builds)


def _place(fn: str, what: str, t: torch.Tensor, dtype, shape, device: int):
    """The address of t, a contiguous tensor of this type and shape on this
    device (else W4A16_ERR_INVALID_ARG)."""
    if (t.dtype is not dtype or t.get_device() != device or t.shape != shape
            or not t.is_contiguous()):
        _refuse(fn, f"{what}: {t.dtype} {tuple(t.shape)} on {t.device}, "
                    f"not contiguous {dtype} {tuple(shape)} on GPU {device}")
    return t.data_ptr()


def _place_rows(fn: str, what: str, t: torch.Tensor, dtype, shape, device: int):
    """(address, row stride) of t, rows of this type and shape with adjacent
    columns on this device (else W4A16_ERR_INVALID_ARG)."""
    if t.dtype is dtype and t.get_device() == device and t.shape == shape:
        if t.is_contiguous():
            return t.data_ptr(), shape[1]
        pitch, step = t.stride()
        if step == 1 or shape[1] == 1:
            return t.data_ptr(), pitch if shape[0] > 1 else max(pitch, shape[1])
    _refuse(fn, f"{what}: {t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}, not rows "
                f"{dtype} {tuple(shape)} on GPU {device}")


def _product(fn: str, call, x, device: int, tokens: int, k: int, columns: int, addend, out,
             out_dtype, stream, weight_at, *last):
    """What both products share: the rows of x [tokens, k], addend and output
    [tokens, columns], and the call. last: the weight's arguments behind its address."""
    if x.dtype is not _BF16:
        _refuse(fn, f"x: {x.dtype}")
    x_stride = k
    if not x.is_contiguous():
        x_stride, step = x.stride()
        if step != 1 and k > 1:
            _refuse(fn, f"x: strides {x.stride()}")
        if tokens <= 1:
            x_stride = max(x_stride, k)
    shape = (tokens, columns)
    if out is None:
        with on_stream(stream):
            out = torch.empty(shape, dtype=out_dtype, device=x.device)
    dtype = out.dtype
    if dtype is not _F32 and dtype is not _BF16:
        _refuse(fn, f"out: {dtype}")
    status = call(
        weight_at, *last, x.data_ptr(), x_stride, tokens,
        None if addend is None else _place(fn, "addend", addend, _F32, shape, device),
        _place(fn, "out", out, dtype, shape, device),
        W4A16_DTYPE_F32 if dtype is _F32 else W4A16_DTYPE_BF16,
        _current_stream(device) if stream is None else stream.cuda_stream)
    if status != W4A16_OK:
        _check(fn, status)
    return out


def _elsewhere(fn: str, x: torch.Tensor):
    """x is not on the current device: the context in which its GPU is."""
    if not x.is_cuda:
        _refuse(fn, f"x: {x.dtype} {tuple(x.shape)} on {x.device}")
    return torch.cuda.device(x.get_device())


def w4a16_linear_few_tokens(x: torch.Tensor, packed: torch.Tensor, n: int,
                            layout: int = W4A16_LAYOUT_KTILE64,
                            addend: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                            out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x . W^T (+ addend FP32 [T, n]) for up to W4A16_FEW_TOKENS_MAX tokens and one
    packed INT4 weight [n, k] (w4a16_prepack of one expert), or, with
    W4A16_LAYOUT_KTILE64_GLU16, silu(x . Wgate^T) * (x . Wup^T), [T, n/2].
    x BF16 [T, k], rows may be strided. out (or out_dtype): FP32 or BF16; out may
    be addend. A blob of another size than [n, k] has is refused."""
    fn = "w4a16_linear_few_tokens"
    device = x.get_device()
    if device < 0 or device != _current_device():
        with _elsewhere(fn, x):
            return w4a16_linear_few_tokens(x, packed, n, layout, addend, out_dtype, out, stream)
    if x.dim() != 2:
        _refuse(fn, f"x {tuple(x.shape)}")
    tokens, k = x.shape
    # 128-row tiles of 64-column steps, 4608 bytes each; with rows that have more or
    # fewer columns than the weight the tiles would be sought at other places
    size = -(-n // 128) * -(-k // 64) * 4608
    at = _blob(fn, "packed", packed, size)
    if packed.numel() != size:
        _refuse(fn, f"packed: {packed.numel()} bytes, a weight [{n}, {k}] has {size}")
    if packed.get_device() != device:
        _refuse(fn, f"x on {x.device}, packed on {packed.device}")
    return _product(fn, load_library().w4a16_linear_few_tokens, x, device, tokens, k,
                    n // 2 if layout == W4A16_LAYOUT_KTILE64_GLU16 else n, addend, out, out_dtype,
                    stream, at, layout, n, k)


def w4a16_dense(x: torch.Tensor, weight: torch.Tensor, gated: bool = False,
                addend: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x . W^T (+ addend FP32 [T, n]) for a BF16 weight [n, k], or, gated (the
    weight's rows are n/2 of the gate, then n/2 of up),
    silu(x . Wgate^T) * (x . Wup^T), [T, n/2]. x BF16 [T, k], rows may be
    strided. out (or out_dtype): FP32 or BF16; out may be addend."""
    fn = "w4a16_dense"
    device = x.get_device()
    if device < 0 or device != _current_device():
        with _elsewhere(fn, x):
            return w4a16_dense(x, weight, gated, addend, out_dtype, out, stream)
    size = weight.shape
    if x.dim() != 2 or len(size) != 2:
        _refuse(fn, f"x {tuple(x.shape)}, weight {tuple(size)}")
    tokens, columns = x.shape
    n, k = size
    if columns != k:
        _refuse(fn, f"x {tuple(x.shape)}, weight {tuple(size)}")
    return _product(fn, load_library().w4a16_dense, x, device, tokens, k, n // 2 if gated else n,
                    addend, out, out_dtype, stream,
                    _place(fn, "weight", weight, _BF16, size, device), n, k, 1 if gated else 0)


def w4a16_dense_info(tokens: int, n: int, k: int, gated: bool = False, out_dtype=torch.bfloat16,
                     at_once=None) -> DenseInfo:
    """How w4a16_dense runs this product on the current device, or on one that runs
    at_once = (pairs, clusters of 1, 2, 4, 8 CTAs) at once."""
    info = DenseInfo()
    counts = None if at_once is None else (_I * 5)(*at_once)
    _check("w4a16_dense_info", load_library().w4a16_dense_info(
        n, k, 1 if gated else 0, tokens,
        W4A16_DTYPE_F32 if out_dtype is _F32 else W4A16_DTYPE_BF16, counts, ctypes.byref(info)))
    return info


def w4a16_block_norm(x: torch.Tensor, pre_weight: Optional[torch.Tensor], eps: float = 1e-6,
                     post_weight: Optional[torch.Tensor] = None,
                     gate: Optional[torch.Tensor] = None,
                     residual: Optional[torch.Tensor] = None, branch_scale: float = 1.0,
                     residual_scale: float = 1.0, weight_offset: float = 0.0,
                     fp8_group: int = W4A16_FP8_NONE, bf16_out: bool = True, out=None,
                     stream=None):
    """p = x * rsqrt(mean(x^2) + eps) * (post_weight + weight_offset) (x itself
    without post_weight), h = residual_scale * residual + branch_scale * gate * p,
    y = h * rsqrt(mean(h^2) + eps) * (pre_weight + weight_offset).
    Returns (bf16(y), bf16(h), e4m3(y * (1 / scale)), scale), the first, third and
    fourth None when not asked for (bf16_out, fp8_group as in
    w4a16_add_rms_norm; pre_weight None: h alone). out: the four tensors to
    write, None for an absent one (it then decides what is written; the second
    may be the residual itself). x FP32 or BF16 [T, H], residual BF16 [T, H], gate
    BF16 [T, H] or [H]; rows may be strided."""
    fn = "w4a16_block_norm"
    device = x.get_device()
    if device < 0 or device != _current_device():
        with _elsewhere(fn, x):
            return w4a16_block_norm(x, pre_weight, eps, post_weight, gate, residual, branch_scale,
                                    residual_scale, weight_offset, fp8_group, bf16_out, out,
                                    stream)
    if x.dim() != 2:
        _refuse(fn, f"x {tuple(x.shape)}")
    rows, hidden = shape = x.shape
    f32 = x.dtype is _F32
    x_at, x_stride = _place_rows(fn, "x", x, _F32 if f32 else _BF16, shape, device)
    post_at = pre_at = r_at = g_at = None
    r_stride = g_stride = 0
    if post_weight is not None:
        post_at = _place(fn, "post_weight", post_weight, _BF16, (hidden,), device)
    if pre_weight is not None:
        pre_at = _place(fn, "pre_weight", pre_weight, _BF16, (hidden,), device)
    if residual is not None:
        r_at, r_stride = _place_rows(fn, "residual", residual, _BF16, shape, device)
    if gate is not None:
        if gate.dim() == 1:
            g_at = _place(fn, "gate", gate, _BF16, (hidden,), device)
        else:
            g_at, g_stride = _place_rows(fn, "gate", gate, _BF16, shape, device)
    groups = 0
    if fp8_group != W4A16_FP8_NONE:
        if fp8_group not in (W4A16_FP8_ROW, W4A16_FP8_GROUP):
            raise W4A16Error(fn, W4A16_ERR_UNSUPPORTED, f"fp8_group {fp8_group}")
        groups = 1 if fp8_group == W4A16_FP8_ROW else -(-hidden // W4A16_FP8_GROUP)
    if out is None:
        normed = pre_weight is not None
        kinds = ((shape, _BF16, bf16_out and normed), (shape, _BF16, True),
                 (shape, _E4M3, fp8_group), ((rows, groups), _F32, fp8_group))
        with on_stream(stream):
            out = tuple(torch.empty(size, dtype=dtype, device=x.device) if wanted else None
                        for size, dtype, wanted in kinds)
    y, h, y8, scales = out
    status = load_library().w4a16_block_norm(
        x_at, W4A16_DTYPE_F32 if f32 else W4A16_DTYPE_BF16, x_stride, post_at, g_at, g_stride,
        r_at, r_stride, pre_at, weight_offset, branch_scale, residual_scale, eps, rows, hidden,
        None if y is None else _place(fn, "out", y, _BF16, shape, device),
        None if h is None else _place(fn, "h_out", h, _BF16, shape, device),
        None if y8 is None else _place(fn, "out_fp8", y8, _E4M3, shape, device),
        None if scales is None else _place(fn, "scales", scales, _F32, (rows, groups), device),
        fp8_group, _current_stream(device) if stream is None else stream.cuda_stream)
    if status != W4A16_OK:
        _check(fn, status)
    return out


def w4a16_read_device_status(workspace: torch.Tensor, stream=None):
    """(status, raw word): W4A16_OK, or W4A16_ERR_TIMEOUT when a wait gave up."""
    detail = _I(0)
    st = load_library().w4a16_read_device_status(_ptr(workspace), ctypes.byref(detail),
                                                 _stream(stream))
    if st not in (W4A16_OK, W4A16_ERR_TIMEOUT):
        _check("w4a16_read_device_status", st)
    return st, int(detail.value)


def w4a16_moe_indexed_gemm_noalloc(mode: int, packed: torch.Tensor, num_experts: int, n: int,
                                   k: int, a: torch.Tensor, tokens: int, topk: int,
                                   sorted_ids: torch.Tensor, expert_ids: torch.Tensor,
                                   num_tokens_padded: torch.Tensor, plan: Plan,
                                   topk_weights: Optional[torch.Tensor] = None,
                                   out: Optional[torch.Tensor] = None, flags: int = 0,
                                   stream=None):
    """w4a16_moe_indexed_gemm for callers that cannot allocate device memory:
    no workspace argument; the library's built-in 32 MiB device array serves
    as the workspace. Only ``out`` is allocated here when the caller passes
    none (a caller that cannot allocate passes its own)."""
    if out is None:
        with on_stream(stream):
            if mode == W4A16_GATE_UP:
                out = torch.empty((tokens * topk, n), dtype=torch.bfloat16, device=a.device)
            else:
                out = torch.empty((tokens, n), dtype=torch.float32, device=a.device)
    _check("w4a16_moe_indexed_gemm_noalloc", load_library().w4a16_moe_indexed_gemm_noalloc(
        mode, _ptr(packed), num_experts, n, k, _ptr(a), tokens, topk, _ptr(sorted_ids),
        _ptr(expert_ids), _ptr(num_tokens_padded), sorted_ids.numel(), _ptr(topk_weights),
        _ptr(out), flags, ctypes.byref(plan), _stream(stream)))
    return out
