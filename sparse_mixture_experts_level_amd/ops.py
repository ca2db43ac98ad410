"""Thin Python binding of libmoe.so (C ABI in include/moe.h).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  Tensors are torch tensors living on the GPU (torch provides device
memory and the current HIP stream); their data pointers are handed to the C
entry points of the same names.  The library must be built
(``python -m sparse_mixture_experts_level_amd.build``); a missing library raises
instead of falling back to anything else.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")
DEBUG_LIB_PATH = os.path.join(_PKG, "libmoe_debug.so")

MOE_NO_CAPACITY = -1
MOE_MAX_EXPERTS = 1024
MOE_OK, MOE_ERR_INVALID, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = range(5)
MOE_DTYPE_F32, MOE_DTYPE_BF16 = 0, 1
MOE_FILL_TOKEN_MAJOR, MOE_FILL_RANK_MAJOR = 0, 1
MOE_OVERFLOW_DROP, MOE_OVERFLOW_REROUTE = 0, 1

SYMBOLS = [
    "moe_capacity", "moe_capacity_topk", "moe_max_rows", "moe_workspace_size", "moe_grouped_gemm_workspace_size",
    "moe_status_string", "moe_last_error", "moe_router_logits", "moe_router_topk",
    "moe_dispatch_permute", "moe_dispatch_reroute", "moe_grouped_swiglu_gemm", "moe_grouped_gate_up_swiglu", "moe_grouped_down",
    "moe_combine_unpermute", "moe_router_aux_loss", "moe_forward", "moe_forward_expert_shard",
    "moe_backward_workspace_size", "moe_backward", "moe_tiled_weights_bytes", "moe_tile_expert_weights",
    "moe_check_topk_ids", "moe_debug_checks", "moe_forward_staged", "moe_forward_noalloc",
    "moe_backward_with_dlogits", "moe_balance_workspace_size", "moe_balance_loss", "moe_balance_loss_backward",
    "moe_grad_norm_workspace_size", "moe_grad_norm", "moe_adamw_check_tensors", "moe_adamw_step",
    "moe_adamw_read_states", "moe_fp8_row_bytes", "moe_fp8_scale_bytes", "moe_quantize_rows_fp8",
    "moe_dequantize_rows_fp8", "moe_fp8_weights_bytes", "moe_fp8_weight_scales_bytes", "moe_quantize_weights_fp8",
    "moe_rms_norm", "moe_rms_norm_backward_workspace_size", "moe_rms_norm_backward",
    "moe_grouped_linear_fp8_workspace_size", "moe_grouped_linear_fp8", "moe_grouped_swiglu_gemm_fp8_workspace_size",
    "moe_grouped_swiglu_gemm_fp8", "moe_forward_fp8_workspace_size", "moe_forward_fp8",
]
MOE_MAX_SEQS = 65536
MOE_ADAMW_BLOCK = 256
MOE_FP8_BLOCK = 128
MOE_NORM_MAX_WIDTH = 32768
MOE_NOALLOC_WORKSPACE_BYTES = 128 << 20

# moe_stage: the stages moe_forward_staged marks, in launch order
STAGES = ["router", "dispatch", "pack_rows", "gate_up", "gate_up_tails", "down", "down_tails", "shared_pack_rows",
          "shared_gate_up", "shared_gate_up_tails", "shared_down", "shared_down_tails", "combine"]


class MoEError(RuntimeError):
    def __init__(self, status: int, func: str, detail: str):
        super().__init__(f"{func} failed: {detail} (status {status})")
        self.status = status


class MoeDesc(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("capacity", ctypes.c_int32),
                ("d_ff_shared", ctypes.c_int32), ("dtype", ctypes.c_int32), ("fill_order", ctypes.c_int32),
                ("overflow", ctypes.c_int32)]


class MoeWeights(ctypes.Structure):
    _fields_ = [("w_router", ctypes.c_void_p), ("w_gate_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("w_shared_gate_up", ctypes.c_void_p), ("w_shared_down", ctypes.c_void_p),
                ("w_gate_up_tiled", ctypes.c_void_p), ("w_down_tiled", ctypes.c_void_p),
                ("w_shared_gate_up_tiled", ctypes.c_void_p), ("w_shared_down_tiled", ctypes.c_void_p)]


class MoeGrads(ctypes.Structure):
    _fields_ = [("dw_router", ctypes.c_void_p), ("dw_gate_up", ctypes.c_void_p), ("dw_down", ctypes.c_void_p),
                ("dw_shared_gate_up", ctypes.c_void_p), ("dw_shared_down", ctypes.c_void_p)]


class MoeRouting(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("topk_ids", ctypes.c_void_p), ("topk_gates", ctypes.c_void_p),
                ("expert_counts", ctypes.c_void_p), ("expert_offsets", ctypes.c_void_p), ("slot", ctypes.c_void_p),
                ("row_token", ctypes.c_void_p), ("assigned_ids", ctypes.c_void_p)]


class MoeFp8Matrix(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


class MoeWeightsFp8(ctypes.Structure):
    _fields_ = [("w_router", ctypes.c_void_p), ("gate_up", MoeFp8Matrix), ("down", MoeFp8Matrix),
                ("shared_gate_up", MoeFp8Matrix), ("shared_down", MoeFp8Matrix)]


class MoeGradView(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class MoeAdamwTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n", ctypes.c_int64), ("param_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("state_bits", ctypes.c_int32), ("weight_decay", ctypes.c_float)]


class MoeAdamwHparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int64), ("lr_dev", ctypes.c_void_p),
                ("step_dev", ctypes.c_void_p), ("norm", ctypes.c_void_p), ("skipped", ctypes.c_void_p)]


_lib = None
_debug_lib = None


def lib() -> ctypes.CDLL:
    """Loads libmoe.so once; raises if it has not been built."""
    global _lib
    if _lib is None:
        _lib = _load(LIB_PATH)
    return _lib


def debug_lib() -> ctypes.CDLL:
    """Loads libmoe_debug.so (the same kernels; host checks of device-side preconditions)."""
    global _debug_lib
    if _debug_lib is None:
        _debug_lib = _load(DEBUG_LIB_PATH)
    return _debug_lib


def _load(path: str) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m sparse_mixture_experts_level_amd.build`")
    L = ctypes.CDLL(path)
    vp, i32, i64, sz, st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    dp = ctypes.POINTER(MoeDesc)
    L.moe_capacity.argtypes, L.moe_capacity.restype = [i32, i32, ctypes.c_double], i32
    L.moe_capacity_topk.argtypes, L.moe_capacity_topk.restype = [i32, i32, i32, ctypes.c_double], i32
    L.moe_max_rows.argtypes, L.moe_max_rows.restype = [dp], i64
    L.moe_workspace_size.argtypes, L.moe_workspace_size.restype = [dp], sz
    L.moe_grouped_gemm_workspace_size.argtypes, L.moe_grouped_gemm_workspace_size.restype = [i32, i64, i32, i32], sz
    L.moe_status_string.argtypes, L.moe_status_string.restype = [st], ctypes.c_char_p
    L.moe_last_error.argtypes, L.moe_last_error.restype = [], ctypes.c_char_p
    L.moe_router_logits.argtypes, L.moe_router_logits.restype = [dp, vp, vp, vp, vp, vp], st
    L.moe_router_topk.argtypes, L.moe_router_topk.restype = [dp, vp, vp, vp, vp], st
    L.moe_dispatch_permute.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_dispatch_permute.restype = st
    L.moe_dispatch_reroute.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_dispatch_reroute.restype = st
    L.moe_grouped_swiglu_gemm.argtypes = [i32, i64, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_grouped_swiglu_gemm.restype = st
    L.moe_grouped_gate_up_swiglu.argtypes = [i32, i64, i32, i32, i32, i32, vp, vp, i64, vp, vp, vp, vp]
    L.moe_grouped_gate_up_swiglu.restype = st
    L.moe_grouped_down.argtypes = [i32, i64, i32, i32, i32, i32, vp, vp, vp, vp, vp]
    L.moe_grouped_down.restype = st
    L.moe_combine_unpermute.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_combine_unpermute.restype = st
    L.moe_router_aux_loss.argtypes = [dp, vp, vp, ctypes.c_float, vp, vp, sz, vp]
    L.moe_router_aux_loss.restype = st
    L.moe_forward.argtypes = [dp, ctypes.POINTER(MoeWeights), vp, vp, vp, ctypes.POINTER(MoeRouting), vp, sz, vp]
    L.moe_forward.restype = st
    L.moe_forward_staged.argtypes = [dp, ctypes.POINTER(MoeWeights), vp, vp, vp, ctypes.POINTER(MoeRouting), vp, sz,
                                     vp, ctypes.POINTER(vp)]
    L.moe_forward_staged.restype = st
    L.moe_forward_noalloc.argtypes = [dp, ctypes.POINTER(MoeWeights), vp, vp, vp, ctypes.POINTER(MoeRouting), vp]
    L.moe_forward_noalloc.restype = st
    L.moe_forward_expert_shard.argtypes = [dp, ctypes.POINTER(MoeWeights), i32, i32, i32, vp, vp, vp,
                                           ctypes.POINTER(MoeRouting), vp, sz, vp]
    L.moe_forward_expert_shard.restype = st
    L.moe_backward_workspace_size.argtypes, L.moe_backward_workspace_size.restype = [dp], sz
    L.moe_backward.argtypes = [dp, ctypes.POINTER(MoeWeights), vp, ctypes.POINTER(MoeRouting), vp, vp,
                               ctypes.POINTER(MoeGrads), vp, sz, vp]
    L.moe_backward.restype = st
    L.moe_tiled_weights_bytes.argtypes, L.moe_tiled_weights_bytes.restype = [dp, i32, i32], sz
    L.moe_tile_expert_weights.argtypes = [dp, i32, vp, vp, vp, vp, vp]
    L.moe_tile_expert_weights.restype = st
    L.moe_check_topk_ids.argtypes, L.moe_check_topk_ids.restype = [dp, vp], st
    L.moe_debug_checks.argtypes, L.moe_debug_checks.restype = [], i32
    f32, gp, tp = ctypes.c_float, ctypes.POINTER(MoeGradView), ctypes.POINTER(MoeAdamwTensor)
    L.moe_backward_with_dlogits.argtypes = [dp, ctypes.POINTER(MoeWeights), vp, ctypes.POINTER(MoeRouting), vp, vp, vp,
                                            ctypes.POINTER(MoeGrads), vp, sz, vp]
    L.moe_backward_with_dlogits.restype = st
    L.moe_balance_workspace_size.argtypes, L.moe_balance_workspace_size.restype = [dp, i32], sz
    L.moe_balance_loss.argtypes = [dp, vp, vp, vp, vp, i32, f32, f32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_balance_loss.restype = st
    L.moe_balance_loss_backward.argtypes = [dp, vp, vp, vp, i32, vp, vp, f32, f32, vp, vp, vp]
    L.moe_balance_loss_backward.restype = st
    L.moe_grad_norm_workspace_size.argtypes, L.moe_grad_norm_workspace_size.restype = [gp, i32], sz
    L.moe_grad_norm.argtypes, L.moe_grad_norm.restype = [gp, i32, f32, vp, vp, sz, vp], st
    L.moe_adamw_check_tensors.argtypes, L.moe_adamw_check_tensors.restype = [tp, i32], st
    L.moe_adamw_step.argtypes, L.moe_adamw_step.restype = [tp, i32, ctypes.POINTER(MoeAdamwHparams), vp], st
    L.moe_adamw_read_states.argtypes = [tp, i32, ctypes.POINTER(vp), ctypes.POINTER(vp), vp]
    L.moe_adamw_read_states.restype = st
    L.moe_fp8_row_bytes.argtypes, L.moe_fp8_row_bytes.restype = [i32], i32
    L.moe_fp8_scale_bytes.argtypes, L.moe_fp8_scale_bytes.restype = [i32], i32
    L.moe_quantize_rows_fp8.argtypes, L.moe_quantize_rows_fp8.restype = [i64, i32, i32, vp, vp, vp, vp], st
    L.moe_dequantize_rows_fp8.argtypes, L.moe_dequantize_rows_fp8.restype = [i64, i32, i32, vp, vp, vp, vp], st
    L.moe_fp8_weights_bytes.argtypes, L.moe_fp8_weights_bytes.restype = [i32, i32, i32, i32], sz
    L.moe_fp8_weight_scales_bytes.argtypes, L.moe_fp8_weight_scales_bytes.restype = [i32, i32, i32, i32], sz
    L.moe_quantize_weights_fp8.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp, vp]
    L.moe_quantize_weights_fp8.restype = st
    L.moe_rms_norm.argtypes, L.moe_rms_norm.restype = [i32, i32, i32, vp, vp, vp, f32, vp, vp, vp, vp, vp, vp], st
    L.moe_rms_norm_backward_workspace_size.argtypes = [i32, i32]
    L.moe_rms_norm_backward_workspace_size.restype = sz
    L.moe_rms_norm_backward.argtypes = [i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_rms_norm_backward.restype = st
    L.moe_grouped_linear_fp8_workspace_size.argtypes = [i32, i64, i32, i32, i32]
    L.moe_grouped_linear_fp8_workspace_size.restype = sz
    L.moe_grouped_linear_fp8.argtypes = [i32, i64, i32, i32, i32, vp, vp, vp, i64, vp, vp, vp, vp, vp, sz, vp]
    L.moe_grouped_linear_fp8.restype = st
    L.moe_grouped_swiglu_gemm_fp8_workspace_size.argtypes = [i32, i64, i32, i32, i32]
    L.moe_grouped_swiglu_gemm_fp8_workspace_size.restype = sz
    L.moe_grouped_swiglu_gemm_fp8.argtypes = [i32, i64, i32, i32, i32, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_grouped_swiglu_gemm_fp8.restype = st
    L.moe_forward_fp8_workspace_size.argtypes, L.moe_forward_fp8_workspace_size.restype = [dp], sz
    L.moe_forward_fp8.argtypes = [dp, ctypes.POINTER(MoeWeightsFp8), vp, vp, vp, vp, vp, ctypes.POINTER(MoeRouting), vp,
                                  sz, vp]
    L.moe_forward_fp8.restype = st
    return L


def _check(status: int, func: str, L=None) -> None:
    if status != MOE_OK:
        L = L or lib()
        raise MoEError(status, func, L.moe_last_error().decode() or L.moe_status_string(status).decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe must be contiguous")
    return t.data_ptr()


_have_gpu = False


def _device() -> int:
    """The current GPU; -2 without one (no tensor's device)."""
    global _have_gpu
    if not _have_gpu:
        _have_gpu = torch.cuda.is_available()
    return torch.cuda.current_device() if _have_gpu else -2


# the current stream's handle without building a torch.cuda.Stream (0.1 instead of 2.7 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream
    dev = _device()
    if dev < 0:
        return None
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream


def _on(stream):
    """The context in which `stream` (a torch stream, a raw handle or None) is torch's current one."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(stream))


def dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return MOE_DTYPE_F32
    if dt == torch.bfloat16:
        return MOE_DTYPE_BF16
    raise ValueError(f"unsupported dtype {dt}")


_FILL = {"token": MOE_FILL_TOKEN_MAJOR, "rank": MOE_FILL_RANK_MAJOR, "slot": MOE_FILL_RANK_MAJOR}
_OVERFLOW = {"drop": MOE_OVERFLOW_DROP, "reroute": MOE_OVERFLOW_REROUTE}


def make_desc(num_tokens, d_model, d_ff, num_experts, top_k, capacity, d_ff_shared=0, dtype=torch.bfloat16,
              fill_order="token", overflow="drop") -> MoeDesc:
    fo = _FILL[fill_order] if isinstance(fill_order, str) else int(fill_order)
    ov = _OVERFLOW[overflow] if isinstance(overflow, str) else int(overflow)
    return MoeDesc(int(num_tokens), int(d_model), int(d_ff), int(num_experts), int(top_k),
                   MOE_NO_CAPACITY if capacity is None else int(capacity), int(d_ff_shared),
                   dtype_code(dtype) if isinstance(dtype, torch.dtype) else int(dtype), fo, ov)


# ------------------------------------------------------------------------ host helpers

def moe_capacity(num_tokens: int, num_experts: int, capacity_factor: Optional[float]) -> Optional[int]:
    c = lib().moe_capacity(int(num_tokens), int(num_experts), 0.0 if capacity_factor is None else float(capacity_factor))
    return None if c == MOE_NO_CAPACITY else int(c)


def moe_capacity_topk(num_tokens: int, num_experts: int, top_k: int,
                      capacity_factor: Optional[float]) -> Optional[int]:
    c = lib().moe_capacity_topk(int(num_tokens), int(num_experts), int(top_k),
                                0.0 if capacity_factor is None else float(capacity_factor))
    return None if c == MOE_NO_CAPACITY else int(c)


def moe_max_rows(desc: MoeDesc) -> int:
    return int(lib().moe_max_rows(ctypes.byref(desc)))


def moe_workspace_size(desc: MoeDesc) -> int:
    return int(lib().moe_workspace_size(ctypes.byref(desc)))


def moe_grouped_gemm_workspace_size(num_groups: int, rows_max: int, d_ff: int, dtype) -> int:
    code = dtype_code(dtype) if isinstance(dtype, torch.dtype) else int(dtype)
    return int(lib().moe_grouped_gemm_workspace_size(int(num_groups), int(rows_max), int(d_ff), code))


def moe_check_topk_ids(desc: MoeDesc, topk_ids_host, L=None) -> None:
    """Host check of the ids precondition on a host int32 [T, k] array (numpy or CPU tensor)."""
    import numpy as np

    a = np.ascontiguousarray(topk_ids_host.numpy() if isinstance(topk_ids_host, torch.Tensor) else topk_ids_host,
                             dtype=np.int32)
    L = L or lib()
    _check(L.moe_check_topk_ids(ctypes.byref(desc), a.ctypes.data_as(ctypes.c_void_p)), "moe_check_topk_ids", L)


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------------ hot path

def moe_router_logits(desc, x, w_router, logit_offset, logits, stream=None) -> None:
    _check(lib().moe_router_logits(ctypes.byref(desc), _ptr(x), _ptr(w_router), _ptr(logit_offset), _ptr(logits),
                                   _stream(stream)), "moe_router_logits")


def moe_router_topk(desc, logits, topk_ids, topk_gates, stream=None) -> None:
    _check(lib().moe_router_topk(ctypes.byref(desc), _ptr(logits), _ptr(topk_ids), _ptr(topk_gates),
                                 _stream(stream)), "moe_router_topk")


def moe_dispatch_permute(desc, topk_ids, x, expert_counts, expert_offsets, slot, row_token, x_perm, ws,
                         stream=None, L=None) -> None:
    L = L or lib()
    _check(L.moe_dispatch_permute(ctypes.byref(desc), _ptr(topk_ids), _ptr(x), _ptr(expert_counts),
                                      _ptr(expert_offsets), _ptr(slot), _ptr(row_token), _ptr(x_perm), _ptr(ws),
                                      0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)),
           "moe_dispatch_permute", L)


def moe_dispatch_reroute(desc, logits, topk_ids, expert_counts, expert_offsets, slot, assigned_ids, row_token, ws,
                         stream=None) -> None:
    _check(lib().moe_dispatch_reroute(ctypes.byref(desc), _ptr(logits), _ptr(topk_ids), _ptr(expert_counts),
                                      _ptr(expert_offsets), _ptr(slot), _ptr(assigned_ids), _ptr(row_token),
                                      _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                      _stream(stream)),
           "moe_dispatch_reroute")


def moe_grouped_swiglu_gemm(num_groups, rows_max, group_rows_max, d_model, d_ff, dtype, x_rows, group_offsets,
                            w_gate_up, w_down, y_rows, ws, stream=None) -> None:
    code = dtype_code(dtype) if isinstance(dtype, torch.dtype) else int(dtype)
    _check(lib().moe_grouped_swiglu_gemm(int(num_groups), int(rows_max), int(group_rows_max), int(d_model), int(d_ff),
                                         code, _ptr(x_rows), _ptr(group_offsets), _ptr(w_gate_up), _ptr(w_down),
                                         _ptr(y_rows), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                         _stream(stream)), "moe_grouped_swiglu_gemm")


def moe_grouped_gate_up_swiglu(num_groups, rows_max, group_rows_max, d_model, d_ff, dtype, x_rows, group_offsets,
                               w_gate_up, h_rows, row_index=None, stream=None) -> None:
    code = dtype_code(dtype) if isinstance(dtype, torch.dtype) else int(dtype)
    n_x = 0 if row_index is None else x_rows.shape[0]
    _check(lib().moe_grouped_gate_up_swiglu(int(num_groups), int(rows_max), int(group_rows_max), int(d_model),
                                            int(d_ff), code, _ptr(x_rows), _ptr(row_index), int(n_x),
                                            _ptr(group_offsets), _ptr(w_gate_up), _ptr(h_rows), _stream(stream)),
           "moe_grouped_gate_up_swiglu")


def moe_grouped_down(num_groups, rows_max, group_rows_max, d_model, d_ff, dtype, h_rows, group_offsets, w_down,
                     y_rows, stream=None) -> None:
    code = dtype_code(dtype) if isinstance(dtype, torch.dtype) else int(dtype)
    _check(lib().moe_grouped_down(int(num_groups), int(rows_max), int(group_rows_max), int(d_model), int(d_ff), code,
                                  _ptr(h_rows), _ptr(group_offsets), _ptr(w_down), _ptr(y_rows), _stream(stream)),
           "moe_grouped_down")


def moe_combine_unpermute(desc, y_perm, topk_ids, topk_gates, slot, expert_offsets, shared_out, out,
                          stream=None, L=None) -> None:
    L = L or lib()
    _check(L.moe_combine_unpermute(ctypes.byref(desc), _ptr(y_perm), _ptr(topk_ids), _ptr(topk_gates), _ptr(slot),
                                   _ptr(expert_offsets), _ptr(shared_out), _ptr(out), _stream(stream)),
           "moe_combine_unpermute", L)


def moe_router_aux_loss(desc, logits, expert_counts, alpha, loss, ws, stream=None) -> None:
    _check(lib().moe_router_aux_loss(ctypes.byref(desc), _ptr(logits), _ptr(expert_counts), float(alpha), _ptr(loss),
                                     _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)),
           "moe_router_aux_loss")


def moe_tiled_weights_bytes(desc, num_experts: int, which: int) -> int:
    return int(lib().moe_tiled_weights_bytes(ctypes.byref(desc), int(num_experts), int(which)))


def moe_tile_expert_weights(desc, num_experts, w_gate_up, w_down, w_gate_up_tiled, w_down_tiled,
                            stream=None) -> None:
    _check(lib().moe_tile_expert_weights(ctypes.byref(desc), int(num_experts), _ptr(w_gate_up), _ptr(w_down),
                                         _ptr(w_gate_up_tiled), _ptr(w_down_tiled), _stream(stream)),
           "moe_tile_expert_weights")


def tiled_weights(desc, w_gate_up, w_down, stream=None):
    """The tile-major copies of w_gate_up [n, 2f, d] and w_down [n, d, f] (bf16, n experts),
    allocated here as uint8 tensors and written by moe_tile_expert_weights."""
    n = w_gate_up.shape[0]
    gu = torch.empty(moe_tiled_weights_bytes(desc, n, 0), dtype=torch.uint8, device=w_gate_up.device)
    dn = torch.empty(moe_tiled_weights_bytes(desc, n, 1), dtype=torch.uint8, device=w_down.device)
    moe_tile_expert_weights(desc, n, w_gate_up, w_down, gu, dn, stream=stream)
    return gu, dn


def _shared_desc(desc) -> MoeDesc:
    """The shared expert as a layer of one expert of width d_ff_shared."""
    one = MoeDesc(**{n: getattr(desc, n) for n, _ in MoeDesc._fields_})
    one.num_experts, one.top_k, one.d_ff, one.d_ff_shared, one.capacity = 1, 1, desc.d_ff_shared, 0, MOE_NO_CAPACITY
    return one


def tiled_shared_weights(desc, w_shared_gate_up, w_shared_down, stream=None):
    """The tile-major copies of the shared expert's [2 f_s, d] and [d, f_s] weights: one expert
    of width d_ff_shared."""
    return tiled_weights(_shared_desc(desc), w_shared_gate_up.unsqueeze(0), w_shared_down.unsqueeze(0), stream=stream)


def tile_shared_weights(desc, w_shared_gate_up, w_shared_down, w_gate_up_tiled, w_down_tiled, stream=None) -> None:
    """Rewrites the copies that tiled_shared_weights() returned."""
    moe_tile_expert_weights(_shared_desc(desc), 1, w_shared_gate_up.unsqueeze(0), w_shared_down.unsqueeze(0),
                            w_gate_up_tiled, w_down_tiled, stream=stream)


def _weights(w_router, w_gate_up, w_down, w_shared_gate_up, w_shared_down, tiled, shared_tiled=None):
    gu_t, dn_t = tiled if tiled is not None else (None, None)
    sgu_t, sdn_t = shared_tiled if shared_tiled is not None else (None, None)
    return MoeWeights(_ptr(w_router), _ptr(w_gate_up), _ptr(w_down), _ptr(w_shared_gate_up), _ptr(w_shared_down),
                      _ptr(gu_t), _ptr(dn_t), _ptr(sgu_t), _ptr(sdn_t))


def moe_forward(desc, w_router, w_gate_up, w_down, x, logit_offset, out, ws, routing: Optional[dict] = None,
                w_shared_gate_up=None, w_shared_down=None, stream=None, tiled=None, shared_tiled=None) -> None:
    """tiled / shared_tiled: optional tile-major copies from tiled_weights() / tiled_shared_weights()."""
    W = _weights(w_router, w_gate_up, w_down, w_shared_gate_up, w_shared_down, tiled, shared_tiled)
    R = None
    if routing is not None:
        R = MoeRouting(*(_ptr(routing.get(n)) for n, _ in MoeRouting._fields_))
    _check(lib().moe_forward(ctypes.byref(desc), ctypes.byref(W), _ptr(x), _ptr(logit_offset), _ptr(out),
                             ctypes.byref(R) if R is not None else None, _ptr(ws),
                             0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)), "moe_forward")


def moe_forward_noalloc(desc, w_router, w_gate_up, w_down, x, logit_offset, out, routing: Optional[dict] = None,
                        w_shared_gate_up=None, w_shared_down=None, stream=None, tiled=None,
                        shared_tiled=None) -> None:
    """moe_forward with the library's fixed per-GPU scratch array as its workspace."""
    W = _weights(w_router, w_gate_up, w_down, w_shared_gate_up, w_shared_down, tiled, shared_tiled)
    R = None
    if routing is not None:
        R = MoeRouting(*(_ptr(routing.get(n)) for n, _ in MoeRouting._fields_))
    _check(lib().moe_forward_noalloc(ctypes.byref(desc), ctypes.byref(W), _ptr(x), _ptr(logit_offset), _ptr(out),
                                     ctypes.byref(R) if R is not None else None, _stream(stream)),
           "moe_forward_noalloc")


def stage_events():
    """MOE_NUM_STAGES + 1 timing events for moe_forward_staged (torch events, created by
    recording them once on the current stream)."""
    evs = [torch.cuda.Event(enable_timing=True) for _ in range(len(STAGES) + 1)]
    for e in evs:
        e.record()
    return evs


def moe_forward_staged(desc, w_router, w_gate_up, w_down, x, logit_offset, out, ws, events,
                       routing: Optional[dict] = None, w_shared_gate_up=None, w_shared_down=None, stream=None,
                       tiled=None, shared_tiled=None) -> None:
    """moe_forward with events[s + 1] recorded after stage s (events from stage_events())."""
    W = _weights(w_router, w_gate_up, w_down, w_shared_gate_up, w_shared_down, tiled, shared_tiled)
    R = None
    if routing is not None:
        R = MoeRouting(*(_ptr(routing.get(n)) for n, _ in MoeRouting._fields_))
    if len(events) != len(STAGES) + 1:
        raise ValueError(f"moe_forward_staged needs {len(STAGES) + 1} events")
    evs = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check(lib().moe_forward_staged(ctypes.byref(desc), ctypes.byref(W), _ptr(x), _ptr(logit_offset), _ptr(out),
                                    ctypes.byref(R) if R is not None else None, _ptr(ws),
                                    0 if ws is None else ws.numel() * ws.element_size(), _stream(stream), evs),
           "moe_forward_staged")


def moe_forward_expert_shard(desc, w_router, w_gate_up_local, w_down_local, expert_begin, expert_end, add_shared, x,
                             logit_offset, out_partial, ws, routing: Optional[dict] = None, w_shared_gate_up=None,
                             w_shared_down=None, stream=None, tiled=None, shared_tiled=None) -> None:
    W = _weights(w_router, w_gate_up_local, w_down_local, w_shared_gate_up, w_shared_down, tiled, shared_tiled)
    R = None
    if routing is not None:
        R = MoeRouting(*(_ptr(routing.get(n)) for n, _ in MoeRouting._fields_))
    _check(lib().moe_forward_expert_shard(ctypes.byref(desc), ctypes.byref(W), int(expert_begin), int(expert_end),
                                          int(bool(add_shared)), _ptr(x), _ptr(logit_offset), _ptr(out_partial),
                                          ctypes.byref(R) if R is not None else None, _ptr(ws),
                                          0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)),
           "moe_forward_expert_shard")


def moe_backward_workspace_size(desc: MoeDesc) -> int:
    return int(lib().moe_backward_workspace_size(ctypes.byref(desc)))


def moe_backward(desc, w_router, w_gate_up, w_down, x, routing: dict, dy, dx, grads: dict, ws,
                 w_shared_gate_up=None, w_shared_down=None, stream=None, tiled=None, shared_tiled=None,
                 dlogits=None) -> None:
    """dlogits: a gradient [T, E] float on the router's logits (moe_balance_loss) to add to the
    gates' (moe_backward_with_dlogits)."""
    W = _weights(w_router, w_gate_up, w_down, w_shared_gate_up, w_shared_down, tiled, shared_tiled)
    R = MoeRouting(*(_ptr(routing.get(n)) for n, _ in MoeRouting._fields_))
    G = MoeGrads(*(_ptr(grads.get(n)) for n, _ in MoeGrads._fields_))
    if dlogits is not None:
        _tensor(dlogits, "dlogits", torch.float32, (desc.num_tokens, desc.num_experts))
        _check(lib().moe_backward_with_dlogits(ctypes.byref(desc), ctypes.byref(W), _ptr(x), ctypes.byref(R), _ptr(dy),
                                               _ptr(dlogits), _ptr(dx), ctypes.byref(G), _ptr(ws),
                                               0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)),
               "moe_backward_with_dlogits")
        return
    _check(lib().moe_backward(ctypes.byref(desc), ctypes.byref(W), _ptr(x), ctypes.byref(R), _ptr(dy), _ptr(dx),
                              ctypes.byref(G), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                              _stream(stream)),
           "moe_backward")


# ------------------------------------------------------------------- balance loss with gradient

def _tensor(t, name: str, dtypes, shape=None, dev=None):
    """Data pointer of a contiguous tensor of one of `dtypes` (and of `shape`) on the current
    GPU (`dev`, where the caller has it); None stays None."""
    if t is None:
        return None
    dt = t.dtype
    if (dt is dtypes or (type(dtypes) is tuple and dt in dtypes)) and (shape is None or t.shape == shape) \
            and t.is_contiguous() and t.get_device() == (_device() if dev is None else dev):
        return t.data_ptr()
    if dt is not dtypes and not (isinstance(dtypes, tuple) and dt in dtypes):
        raise ValueError(f"{name} has dtype {dt}, expected {dtypes}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}; the library runs on the current GPU")


def _num_seqs(seq_offsets) -> int:
    return 1 if seq_offsets is None else seq_offsets.numel() - 1


def moe_balance_workspace_size(desc: MoeDesc, num_seqs: int = 1) -> int:
    return int(lib().moe_balance_workspace_size(ctypes.byref(desc), int(num_seqs)))


def moe_balance_loss(desc, logits, topk_ids, alpha, z_coeff, counts, seq_tokens, mean_probs, losses, ws,
                     token_mask=None, seq_offsets=None, dlogits=None, stream=None) -> None:
    """counts [S, E] int32, seq_tokens [S] int32, mean_probs [S, E], losses [2] (balance, z) and, if
    given, dlogits [T, E] are written; S = 1, or seq_offsets.numel() - 1."""
    T, E, k, S = desc.num_tokens, desc.num_experts, desc.top_k, _num_seqs(seq_offsets)
    dev = _device()
    _check(lib().moe_balance_loss(
        ctypes.byref(desc), _tensor(logits, "logits", torch.float32, (T, E), dev),
        _tensor(topk_ids, "topk_ids", torch.int32, (T, k), dev),
        _tensor(token_mask, "token_mask", (torch.uint8, torch.bool), (T,), dev),
        _tensor(seq_offsets, "seq_offsets", torch.int32, (S + 1,), dev), S, alpha, z_coeff,
        _tensor(counts, "counts", torch.int32, (S, E), dev), _tensor(seq_tokens, "seq_tokens", torch.int32, (S,), dev),
        _tensor(mean_probs, "mean_probs", torch.float32, (S, E), dev),
        _tensor(losses, "losses", torch.float32, (2,), dev), _tensor(dlogits, "dlogits", torch.float32, (T, E), dev),
        _tensor(ws, "ws", torch.uint8, None, dev), 0 if ws is None else ws.numel(), _stream(stream)),
        "moe_balance_loss")


def moe_balance_loss_backward(desc, logits, counts, seq_tokens, alpha, z_coeff, dlogits, token_mask=None,
                              seq_offsets=None, dloss=None, stream=None) -> None:
    """dlogits from the forward's counts and seq_tokens; dloss [2]: upstream gradients (None: ones)."""
    T, E, S = desc.num_tokens, desc.num_experts, _num_seqs(seq_offsets)
    dev = _device()
    _check(lib().moe_balance_loss_backward(
        ctypes.byref(desc), _tensor(logits, "logits", torch.float32, (T, E), dev),
        _tensor(token_mask, "token_mask", (torch.uint8, torch.bool), (T,), dev),
        _tensor(seq_offsets, "seq_offsets", torch.int32, (S + 1,), dev), S,
        _tensor(counts, "counts", torch.int32, (S, E), dev), _tensor(seq_tokens, "seq_tokens", torch.int32, (S,), dev),
        alpha, z_coeff, _tensor(dloss, "dloss", torch.float32, (2,), dev),
        _tensor(dlogits, "dlogits", torch.float32, (T, E), dev), _stream(stream)), "moe_balance_loss_backward")


# --------------------------------------------------------------- gradient norm and AdamW step

class GradList:
    """Gradient tensors with the host array of views that moe_grad_norm takes (grad_list()).

    The list stands for the memory that the tensors have when it is built, and keeps it alive:
    write gradients in place, or build the list again."""

    def __init__(self, grads):
        self.grads = [g.detach() for g in grads]
        self.views = (MoeGradView * max(len(self.grads), 1))()
        self.device = _device()
        for i, g in enumerate(self.grads):
            self.views[i] = MoeGradView(_tensor(g, f"grads[{i}]", (torch.float32, torch.bfloat16), None, self.device),
                                        g.numel(), dtype_code(g.dtype), 0)

    def __len__(self):
        return len(self.grads)


def grad_list(grads) -> GradList:
    return GradList(grads)


def moe_grad_norm_workspace_size(grads: GradList) -> int:
    return int(lib().moe_grad_norm_workspace_size(grads.views, len(grads)))


def moe_grad_norm(grads: GradList, max_norm: float, out, ws, stream=None) -> None:
    """out [2] float: the norm over every gradient (infinity past the floats), and min(1, max_norm / (norm +
    1e-6)), NaN where a gradient is not finite."""
    dev = _device()
    if dev != grads.device:
        raise RuntimeError(f"the gradients are on GPU {grads.device}, which is not the current one")
    _check(lib().moe_grad_norm(grads.views, len(grads), max_norm, _tensor(out, "out", torch.float32, (2,), dev),
                               _tensor(ws, "ws", torch.uint8, None, dev), 0 if ws is None else ws.numel(),
                               _stream(stream)), "moe_grad_norm")


def moe_adamw_check_tensors(tensors, num_tensors: int) -> None:
    _check(lib().moe_adamw_check_tensors(tensors, int(num_tensors)), "moe_adamw_check_tensors")


def moe_adamw_step(tensors, num_tensors: int, hparams: MoeAdamwHparams, stream=None) -> None:
    _check(lib().moe_adamw_step(tensors, num_tensors, ctypes.byref(hparams), _stream(stream)), "moe_adamw_step")


def moe_adamw_read_states(tensors, num_tensors: int, m_out=None, v_out=None, stream=None) -> None:
    """m_out, v_out: per tensor a float tensor or None; None: not wanted."""
    def pointers(outs, name):
        if outs is None:
            return None
        if len(outs) != num_tensors:
            raise ValueError(f"{name} holds {len(outs)} tensors, expected {num_tensors}")
        ptrs = (ctypes.c_void_p * max(num_tensors, 1))()
        for i, o in enumerate(outs):
            if o is not None:
                ptrs[i] = _tensor(o, name, torch.float32, None, dev)
                if o.numel() != tensors[i].n:
                    raise ValueError(f"{name}[{i}] holds {o.numel()} values, expected {tensors[i].n}")
        return ptrs
    dev = _device()
    _check(lib().moe_adamw_read_states(tensors, num_tensors, pointers(m_out, "m_out"), pointers(v_out, "v_out"),
                                       _stream(stream)), "moe_adamw_read_states")


def _capturing(stream) -> bool:
    with _on(stream):
        return torch.cuda.is_current_stream_capturing()


class MoEAdamW:
    """AdamW over a list of parameter tensors with fixed gradient tensors (moe_adamw_step), after
    clipping by the gradients' norm when max_grad_norm is given (moe_grad_norm).

    Parameters and gradients are float or bf16; weight_decay is one value or one per tensor.
    state_bits 32 or 8; with 8 take a beta2 of at most 0.98 (with 0.999 rounding to the nearest code
    keeps v from falling with its own decay; include/moe.h has the borders); master_weights keeps a float copy of each bf16 parameter.  `states`
    (one dict of m, v, m_scale, v_scale, master per tensor) takes existing state tensors
    instead of new zeros: a master in it is used whatever master_weights says, and one that
    master_weights asks for and it lacks is made from the parameter (`optimizer.states` then
    holds it, not the caller's dict).  `step` is the number of updates already done.  With capturable=True
    the step number and lr live on the device, so that a step captured into a HIP graph
    counts on at every replay (step_count only counts calls); set the rate with set_lr() then.
    A step with a gradient that is not finite changes no tensor if max_grad_norm is given: grad_norm[1]
    is NaN then (grad_norm[0] can be infinite for finite gradients, whose step is made).  `skipped`
    counts these steps on the device, and the bias corrections go by the updates made
    (updates_done()).

    Tensors are used on the stream of the call, on the GPU that is current when the optimizer is
    built; allocation happens here, never in step().  The optimizer reads the memory that the
    gradients have when it is built, and keeps it alive: write gradients in place.  A parameter
    or gradient tensor whose memory has been replaced since is refused by step()."""

    def __init__(self, params, grads, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, max_grad_norm=None,
                 state_bits=32, master_weights=False, states=None, step=0, capturable=False):
        self.params, given = list(params), list(grads)
        self.grads = [g.detach() for g in given]
        n = len(self.params)
        if len(self.grads) != n or (states is not None and len(states) != n):
            raise ValueError("params, grads and states must have one entry per tensor")
        if state_bits not in (32, 8):
            raise ValueError(f"state_bits {state_bits}: 32 or 8")
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * n
        if len(decay) != n:
            raise ValueError("weight_decay must be one value or one per tensor")
        self.state_bits, self.max_grad_norm, self.step_count = state_bits, max_grad_norm, int(step)
        self.states = ([self._new_state(p, master_weights) for p in self.params] if states is None else
                       [self._given_state(p, s, master_weights) for p, s in zip(self.params, states)])
        self.tensors = (MoeAdamwTensor * max(n, 1))()
        fp = (torch.float32, torch.bfloat16)
        kinds = (torch.float32, torch.float32) if state_bits == 32 else (torch.int8, torch.uint8)
        for i, (p, g, s) in enumerate(zip(self.params, self.grads, self.states)):
            if p.numel() != g.numel():
                raise ValueError(f"params[{i}] holds {p.numel()} values, grads[{i}] {g.numel()}")
            size, blocks = (p.numel(),), (-(-p.numel() // MOE_ADAMW_BLOCK),)

            def ptr(name, kind, shape):
                t = s.get(name)
                return None if t is None else _tensor(t.view(-1), f"states[{i}].{name}", kind, shape)
            self.tensors[i] = MoeAdamwTensor(
                _tensor(p, f"params[{i}]", fp), _tensor(g, f"grads[{i}]", fp), ptr("master", torch.float32, size),
                ptr("m", kinds[0], size), ptr("v", kinds[1], size),
                ptr("m_scale", torch.float32, blocks) if state_bits == 8 else None,
                ptr("v_scale", torch.float32, blocks) if state_bits == 8 else None,
                p.numel(), dtype_code(p.dtype), dtype_code(g.dtype), state_bits, float(decay[i]))
        moe_adamw_check_tensors(self.tensors, n)
        self._device = _device()
        self._watched = self.params + given  # (a detached tensor keeps the memory it was made with)
        self._pointers = list(map(torch.Tensor.data_ptr, self._watched))
        # what the host array points at stays alive, whatever becomes of the caller's tensors
        self._memory = [t.detach() for s in self.states for t in s.values() if t is not None]
        self._memory += [p.detach() for p in self.params]
        self.hparams = MoeAdamwHparams(float(lr), float(betas[0]), float(betas[1]), float(eps), self.step_count, None,
                                       None, None, None)
        self._check_lr(lr)
        if max_grad_norm is not None and not ctypes.c_float(max_grad_norm).value > 0:
            raise ValueError(f"max_grad_norm {max_grad_norm}: above 0 as a float, or None")
        self.hparams.step += 1
        moe_adamw_step(self.tensors, 0, self.hparams)  # of no tensor: only the checks
        device = self.params[0].device if n else "cuda"
        self.capturable = capturable
        if capturable:
            self.lr_dev = torch.full((1,), float(lr), dtype=torch.float32, device=device)
            self.step_dev = torch.full((1,), self.step_count, dtype=torch.int64, device=device)
            self.hparams.lr_dev, self.hparams.step_dev = self.lr_dev.data_ptr(), self.step_dev.data_ptr()
        self.grad_norm = None  # [2]: the norm before clipping, the factor applied
        self.skipped = None    # [1]: steps left undone for a gradient that was not finite
        if max_grad_norm is not None:
            self._grad_list = grad_list(self.grads)
            self._ws = workspace(moe_grad_norm_workspace_size(self._grad_list), device)
            self.grad_norm = torch.zeros(2, dtype=torch.float32, device=device)
            self.skipped = torch.zeros(1, dtype=torch.int64, device=device)
            self.hparams.norm, self.hparams.skipped = self.grad_norm.data_ptr(), self.skipped.data_ptr()

    def _new_state(self, p, master_weights):
        z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=p.device)  # noqa: E731
        if self.state_bits == 32:
            s = {"m": z(p.shape, torch.float32), "v": z(p.shape, torch.float32)}
        else:
            blocks = -(-p.numel() // MOE_ADAMW_BLOCK)
            s = {"m": z(p.shape, torch.int8), "v": z(p.shape, torch.uint8), "m_scale": z((blocks,), torch.float32),
                 "v_scale": z((blocks,), torch.float32)}
        if master_weights and p.dtype != torch.float32:
            s["master"] = p.detach().float()
        return s

    @staticmethod
    def _given_state(p, s, master_weights):
        if master_weights and p.dtype != torch.float32 and s.get("master") is None:
            s = dict(s, master=p.detach().float())
        return s

    @staticmethod
    def _check_lr(lr):
        if not 0 <= lr < float("inf"):
            raise ValueError(f"lr {lr} must be finite and >= 0")

    def set_lr(self, lr: float) -> None:
        self._check_lr(lr)
        self.hparams.lr = float(lr)
        if self.capturable:
            self.lr_dev.fill_(float(lr))

    def _check_device(self):
        if _device() != self._device:
            raise RuntimeError(f"the optimizer's tensors are on GPU {self._device}, which is not the current one")

    def step(self, stream=None) -> None:
        n = len(self.params)
        self._check_device()
        now = list(map(torch.Tensor.data_ptr, self._watched))
        if now != self._pointers:
            what = "parameter" if now[:n] != self._pointers[:n] else "gradient"
            raise RuntimeError(f"a {what}'s memory has been replaced: build the optimizer again")
        if self.capturable:
            if stream is not None:
                raise ValueError("a capturable step runs on the current stream")
        elif _capturing(stream):
            raise RuntimeError("a captured step would repeat its step number: construct MoEAdamW with capturable=True")
        if self.max_grad_norm is not None:
            moe_grad_norm(self._grad_list, self.max_grad_norm, self.grad_norm, self._ws, stream=stream)
        if self.capturable:  # behind what may refuse the call
            self.step_dev.add_(1)
        self.hparams.step = self.step_count + 1
        moe_adamw_step(self.tensors, n, self.hparams, stream=stream)
        self.step_count += 1

    def updates_done(self) -> int:
        """Steps that updated the tensors, those before `step` included: the `step` to resume with.
        Reads the device (waits for the current stream)."""
        steps = int(self.step_dev) if self.capturable else self.step_count
        return steps - (0 if self.skipped is None else int(self.skipped))

    def read_states(self, m_out=None, v_out=None, stream=None):
        """8-bit states as the floats they stand for, into the given tensors or new ones (which
        belong to `stream`)."""
        self._check_device()
        if m_out is None and v_out is None:
            with _on(stream):
                m_out, v_out = ([torch.empty(p.shape, dtype=torch.float32, device=p.device) for p in self.params]
                                for _ in range(2))
        moe_adamw_read_states(self.tensors, len(self.params), m_out, v_out, stream=stream)
        return m_out, v_out


# ------------------------------------------------- 8-bit floating point, norm, 8-bit experts

_FP = (torch.float32, torch.bfloat16)
_CODES = (torch.uint8, torch.float8_e4m3fn)


def moe_fp8_row_bytes(k: int) -> int:
    return int(lib().moe_fp8_row_bytes(k))


def moe_fp8_scale_bytes(k: int) -> int:
    return int(lib().moe_fp8_scale_bytes(k))


def _rows8(codes, scale, names, rows, k, dev):
    """Pointers of rows in 8 bits: codes [rows, moe_fp8_row_bytes(k)], scale [rows, moe_fp8_scale_bytes(k)]."""
    if codes is None and scale is None:
        return None, None
    blocks = (k + 127) >> 7
    return (_tensor(codes, names[0], _CODES, (rows, blocks << 7), dev),
            _tensor(scale, names[1], torch.uint8, (rows, (blocks + 3) & ~3), dev))


def fp8_rows(rows: int, k: int, device="cuda"):
    """New (codes, scale) for rows of k values in 8 bits."""
    return (torch.empty((rows, moe_fp8_row_bytes(k)), dtype=torch.uint8, device=device),
            torch.empty((rows, moe_fp8_scale_bytes(k)), dtype=torch.uint8, device=device))


def moe_quantize_rows_fp8(x, codes, scale, stream=None) -> None:
    rows, k = x.shape
    dev = _device()
    _check(lib().moe_quantize_rows_fp8(rows, k, dtype_code(x.dtype), _tensor(x, "x", _FP, None, dev),
                                       *_rows8(codes, scale, ("codes", "scale"), rows, k, dev), _stream(stream)),
           "moe_quantize_rows_fp8")


def moe_dequantize_rows_fp8(codes, scale, out, stream=None) -> None:
    rows, k = out.shape
    dev = _device()
    _check(lib().moe_dequantize_rows_fp8(rows, k, dtype_code(out.dtype),
                                         *_rows8(codes, scale, ("codes", "scale"), rows, k, dev),
                                         _tensor(out, "out", _FP, None, dev), _stream(stream)),
           "moe_dequantize_rows_fp8")


def moe_fp8_weights_bytes(num_groups: int, n_out: int, k: int, swiglu: bool) -> int:
    return int(lib().moe_fp8_weights_bytes(int(num_groups), int(n_out), int(k), int(bool(swiglu))))


def moe_fp8_weight_scales_bytes(num_groups: int, n_out: int, k: int, swiglu: bool) -> int:
    return int(lib().moe_fp8_weight_scales_bytes(int(num_groups), int(n_out), int(k), int(bool(swiglu))))


def moe_quantize_weights_fp8(num_groups, n_out, k, swiglu, w, codes, scale, stream=None) -> None:
    """w [G, n_out, k], or with swiglu [G, 2 n_out, k] (gate rows, then up rows), float or bf16."""
    dev = _device()
    _check(lib().moe_quantize_weights_fp8(
        int(num_groups), int(n_out), int(k), int(bool(swiglu)), dtype_code(w.dtype),
        _tensor(w, "w", _FP, (num_groups, n_out * (2 if swiglu else 1), k), dev),
        *_matrix8(codes, scale, "codes", num_groups, n_out, k, swiglu, dev), _stream(stream)), "moe_quantize_weights_fp8")


def _matrix8(codes, scale, name, num_groups, n_out, k, swiglu, dev):
    """Pointers of a matrix in 8 bits, whose tensors must have the sizes of its shape."""
    kb, parts = (k + 127) >> 7, num_groups << 1 if swiglu else num_groups
    return (_tensor(codes, name, torch.uint8, (parts * ((n_out + 15) >> 4) * kb * 2048,), dev),
            _tensor(scale, name + "'s scale", torch.uint8, (parts * ((n_out + 127) >> 7) * ((kb + 3) & ~3),), dev))


def fp8_weights(w, swiglu=False, stream=None):
    """(codes, scale) of w [G, n, k] in 8 bits, allocated here as flat uint8 tensors; swiglu: w is a gate_up matrix."""
    g, n, k = w.shape
    if swiglu and n % 2:
        raise ValueError(f"a gate_up matrix has as many gate as up rows: got {n}")
    n_out = n // 2 if swiglu else n
    with _on(stream):
        codes = torch.empty(moe_fp8_weights_bytes(g, n_out, k, swiglu), dtype=torch.uint8, device=w.device)
        scale = torch.empty(moe_fp8_weight_scales_bytes(g, n_out, k, swiglu), dtype=torch.uint8, device=w.device)
    moe_quantize_weights_fp8(g, n_out, k, swiglu, w, codes, scale, stream=stream)
    return codes, scale


def moe_rms_norm(x, weight, eps, residual=None, h=None, y=None, y8=None, y_scale=None, rstd=None, stream=None) -> None:
    """h = x + residual, rstd [T] float, y = h rstd weight, also in 8 bits (y8, y_scale): what is given is written."""
    T, d = x.shape
    dev, dt, shape = _device(), x.dtype, x.shape
    _check(lib().moe_rms_norm(
        T, d, dtype_code(dt), _tensor(x, "x", _FP, None, dev), _tensor(residual, "residual", dt, shape, dev),
        _tensor(weight, "weight", dt, (d,), dev), eps, _tensor(h, "h", dt, shape, dev), _tensor(y, "y", dt, shape, dev),
        *_rows8(y8, y_scale, ("y8", "y_scale"), T, d, dev), _tensor(rstd, "rstd", torch.float32, (T,), dev),
        _stream(stream)), "moe_rms_norm")


def moe_rms_norm_backward_workspace_size(num_tokens: int, d_model: int) -> int:
    return int(lib().moe_rms_norm_backward_workspace_size(int(num_tokens), int(d_model)))


def moe_rms_norm_backward(dy, h, weight, rstd, dx, dweight, ws, dh=None, stream=None) -> None:
    """dx (of x and of residual) and dweight [d] float from dy, the forward's h and rstd, and dh, the gradient that
    reaches h itself."""
    T, d = h.shape
    dev, dt, shape = _device(), h.dtype, h.shape
    _check(lib().moe_rms_norm_backward(
        T, d, dtype_code(dt), _tensor(dy, "dy", dt, shape, dev), _tensor(h, "h", _FP, None, dev),
        _tensor(weight, "weight", dt, (d,), dev), _tensor(rstd, "rstd", torch.float32, (T,), dev),
        _tensor(dh, "dh", dt, shape, dev), _tensor(dx, "dx", dt, shape, dev),
        _tensor(dweight, "dweight", torch.float32, (d,), dev), _tensor(ws, "ws", torch.uint8, None, dev),
        0 if ws is None else ws.numel(), _stream(stream)), "moe_rms_norm_backward")


def _fp8_operands(num_groups, rows_max, k, x8, x_scale, group_offsets, row_index, dev):
    rows = rows_max if row_index is None else x8.shape[0]
    codes, scale = _rows8(x8, x_scale, ("x8", "x_scale"), rows, k, dev)
    return (codes, scale, _tensor(row_index, "row_index", torch.int32, (rows_max,), dev), rows,
            _tensor(group_offsets, "group_offsets", torch.int32, (num_groups + 1,), dev))


def moe_grouped_linear_fp8_workspace_size(num_groups, rows_max, group_rows_max, n_out, k) -> int:
    return int(lib().moe_grouped_linear_fp8_workspace_size(int(num_groups), int(rows_max), int(group_rows_max),
                                                           int(n_out), int(k)))


def moe_grouped_linear_fp8(num_groups, rows_max, group_rows_max, n_out, k, x8, x_scale, group_offsets, w8, w_scale,
                           y_rows, ws, row_index=None, stream=None) -> None:
    """y_rows[r] = W[g] x8[r] for the rows of each group; w8, w_scale from fp8_weights(w [G, n_out, k])."""
    dev = _device()
    _check(lib().moe_grouped_linear_fp8(
        num_groups, rows_max, group_rows_max, n_out, k,
        *_fp8_operands(num_groups, rows_max, k, x8, x_scale, group_offsets, row_index, dev),
        *_matrix8(w8, w_scale, "w8", num_groups, n_out, k, False, dev),
        _tensor(y_rows, "y_rows", torch.bfloat16, (rows_max, n_out), dev), _tensor(ws, "ws", torch.uint8, None, dev),
        0 if ws is None else ws.numel(), _stream(stream)), "moe_grouped_linear_fp8")


def moe_grouped_swiglu_gemm_fp8_workspace_size(num_groups, rows_max, group_rows_max, d_model, d_ff) -> int:
    return int(lib().moe_grouped_swiglu_gemm_fp8_workspace_size(int(num_groups), int(rows_max), int(group_rows_max),
                                                                int(d_model), int(d_ff)))


def moe_grouped_swiglu_gemm_fp8(num_groups, rows_max, group_rows_max, d_model, d_ff, x8, x_scale, group_offsets,
                                w_gate_up8, w_gate_up_scale, w_down8, w_down_scale, y_rows, ws, row_index=None,
                                stream=None) -> None:
    """The experts' FFN in 8 bits: fp8_weights(w_gate_up, swiglu=True) and fp8_weights(w_down)."""
    dev = _device()
    _check(lib().moe_grouped_swiglu_gemm_fp8(
        num_groups, rows_max, group_rows_max, d_model, d_ff,
        *_fp8_operands(num_groups, rows_max, d_model, x8, x_scale, group_offsets, row_index, dev),
        *_matrix8(w_gate_up8, w_gate_up_scale, "w_gate_up8", num_groups, d_ff, d_model, True, dev),
        *_matrix8(w_down8, w_down_scale, "w_down8", num_groups, d_model, d_ff, False, dev),
        _tensor(y_rows, "y_rows", torch.bfloat16, (rows_max, d_model), dev), _tensor(ws, "ws", torch.uint8, None, dev),
        0 if ws is None else ws.numel(), _stream(stream)), "moe_grouped_swiglu_gemm_fp8")


def moe_forward_fp8_workspace_size(desc: MoeDesc) -> int:
    return int(lib().moe_forward_fp8_workspace_size(ctypes.byref(desc)))


def moe_forward_fp8(desc, w_router, gate_up, down, x, logit_offset, out, ws, routing: Optional[dict] = None,
                    shared_gate_up=None, shared_down=None, x8=None, x_scale=None, stream=None) -> None:
    """moe_forward with experts in 8 bits: gate_up, down (and the shared expert's) are the pairs that fp8_weights()
    returns; x8, x_scale: x in 8 bits, or None (quantised here)."""
    dev, T, d, E, f, fs = _device(), desc.num_tokens, desc.d_model, desc.num_experts, desc.d_ff, desc.d_ff_shared
    m = lambda pair, name, g, n, k, s: (  # noqa: E731
        MoeFp8Matrix(None, None) if pair is None else MoeFp8Matrix(*_matrix8(*pair, name, g, n, k, s, dev)))
    W = MoeWeightsFp8(_tensor(w_router, "w_router", torch.bfloat16, (E, d), dev), m(gate_up, "gate_up", E, f, d, True),
                      m(down, "down", E, d, f, False), m(shared_gate_up, "shared_gate_up", 1, fs, d, True),
                      m(shared_down, "shared_down", 1, d, fs, False))
    R = None
    if routing is not None:
        R = MoeRouting(*(_ptr(routing.get(n)) for n, _ in MoeRouting._fields_))
    _check(lib().moe_forward_fp8(
        ctypes.byref(desc), ctypes.byref(W), _tensor(x, "x", torch.bfloat16, (T, d), dev),
        *_rows8(x8, x_scale, ("x8", "x_scale"), T, d, dev), _tensor(logit_offset, "logit_offset", torch.float32, (E,), dev),
        _tensor(out, "out", torch.bfloat16, (T, d), dev), ctypes.byref(R) if R is not None else None,
        _tensor(ws, "ws", torch.uint8, None, dev), 0 if ws is None else ws.numel(), _stream(stream)), "moe_forward_fp8")


class MoELayer:
    """Holds one layer's device tensors and a workspace, and runs moe_forward.

    fp8: the experts (and the shared expert) in 8 bits, quantised here once (moe_forward_fp8); the bf16 ones of `inputs` are
    not read again: they may be set to None, and where they change a layer has to be built again.
    norm_weight [d]: a norm in front of the layer (moe_rms_norm with norm_eps): forward(residual) takes
    inputs.x + residual, kept in `h` (the next block's residual; a copy of inputs.x without a residual), and the layer runs
    on its norm, `normed`, which it gets in 8 bits too with fp8.

    Convenience only: allocation happens here, once, never inside a forward call."""

    def __init__(self, inputs, capacity, device="cuda", fill_order="token", overflow="drop", tiled=False,
                 shared_tiled=False, fp8=False, norm_weight=None, norm_eps=1e-6):
        w = inputs.workload
        self.inputs = inputs
        self.desc = make_desc(w.num_tokens, w.d_model, w.d_ff, w.num_experts, w.top_k, capacity,
                              w.d_ff_shared, w.torch_dtype, fill_order=fill_order, overflow=overflow)
        if fp8 and (tiled or shared_tiled):
            raise ValueError("tile-major copies are of bf16 weights: not with fp8")
        if fp8 and self.desc.dtype != MOE_DTYPE_BF16:
            raise ValueError("experts in 8 bits are implemented for bf16 layers")
        self.fp8, self.norm_weight, self.norm_eps = None, norm_weight, norm_eps
        if fp8:
            self.fp8 = dict(gate_up=fp8_weights(inputs.w_gate_up, swiglu=True), down=fp8_weights(inputs.w_down))
            if w.d_ff_shared:
                self.fp8.update(shared_gate_up=fp8_weights(inputs.w_shared_gate_up.unsqueeze(0), swiglu=True),
                                shared_down=fp8_weights(inputs.w_shared_down.unsqueeze(0)))
        self.x8 = self.x_scale = None
        if norm_weight is not None:
            self.h, self.normed = torch.empty_like(inputs.x), torch.empty_like(inputs.x)
            self.rstd = torch.empty((w.num_tokens,), dtype=torch.float32, device=device)
            if fp8:
                self.x8, self.x_scale = fp8_rows(w.num_tokens, w.d_model, device)
        self.ws = workspace((moe_forward_fp8_workspace_size if fp8 else moe_workspace_size)(self.desc), device)
        self.out = torch.empty_like(inputs.x)
        T, E, k = w.num_tokens, w.num_experts, w.top_k
        R = moe_max_rows(self.desc)
        i32 = dict(dtype=torch.int32, device=device)
        self.routing = {
            "logits": torch.empty((T, E), dtype=torch.float32, device=device),
            "topk_ids": torch.empty((T, k), **i32),
            "topk_gates": torch.empty((T, k), dtype=torch.float32, device=device),
            "expert_counts": torch.empty((E,), **i32),
            "expert_offsets": torch.empty((E + 1,), **i32),
            "slot": torch.empty((T, k), **i32),
            "row_token": torch.empty((max(R, 1),), **i32),
            "assigned_ids": torch.empty((T, k), **i32),
        }
        # the routed weights' tile-major copies, prepared once (bf16)
        self.tiled = tiled_weights(self.desc, inputs.w_gate_up, inputs.w_down) if tiled else None
        self.shared_tiled = (tiled_shared_weights(self.desc, inputs.w_shared_gate_up, inputs.w_shared_down)
                             if shared_tiled and w.d_ff_shared else None)

    def _layer_input(self, residual, stream):
        """What the layer runs on: inputs.x, or the norm of inputs.x + residual."""
        if self.norm_weight is None:
            if residual is not None:
                raise ValueError("a residual is added by the norm: construct MoELayer with norm_weight")
            return self.inputs.x
        moe_rms_norm(self.inputs.x, self.norm_weight, self.norm_eps, residual=residual, h=self.h, y=self.normed,
                     y8=self.x8, y_scale=self.x_scale, rstd=self.rstd, stream=stream)
        return self.normed

    def forward_staged(self, events, with_routing=False, stream=None):
        if self.fp8 is not None or self.norm_weight is not None:
            raise ValueError("forward_staged times moe_forward: not with fp8 or a norm")
        i = self.inputs
        moe_forward_staged(self.desc, i.w_router, i.w_gate_up, i.w_down, i.x, i.logit_offset, self.out, self.ws,
                           events, routing=self.routing if with_routing else None,
                           w_shared_gate_up=i.w_shared_gate_up, w_shared_down=i.w_shared_down, stream=stream,
                           tiled=self.tiled, shared_tiled=self.shared_tiled)
        return self.out

    def forward(self, with_routing=True, stream=None, residual=None):
        i = self.inputs
        x = self._layer_input(residual, stream)
        if self.fp8 is not None:
            moe_forward_fp8(self.desc, i.w_router, self.fp8["gate_up"], self.fp8["down"], x, i.logit_offset, self.out,
                            self.ws, routing=self.routing if with_routing else None,
                            shared_gate_up=self.fp8.get("shared_gate_up"), shared_down=self.fp8.get("shared_down"),
                            x8=self.x8, x_scale=self.x_scale, stream=stream)
            return self.out
        moe_forward(self.desc, i.w_router, i.w_gate_up, i.w_down, x, i.logit_offset, self.out, self.ws,
                    routing=self.routing if with_routing else None, w_shared_gate_up=i.w_shared_gate_up,
                    w_shared_down=i.w_shared_down, stream=stream, tiled=self.tiled, shared_tiled=self.shared_tiled)
        return self.out


class MoETrainer:
    """One bf16 layer's training step: moe_forward, the balance and z losses with their gradient
    (moe_balance_loss), moe_backward_with_dlogits, the clipped AdamW step, and the tile-major copies
    rewritten from the new weights.

    Buffers are allocated here, once; the optimizer's options (lr, weight_decay, max_grad_norm,
    state_bits, master_weights, capturable, ...) are MoEAdamW's.  The router is not decayed unless
    weight_decay is given per tensor (router, gate_up, down[, shared gate_up, shared down][, norm]).
    norm_weight, norm_eps: a norm in front of the layer, as MoELayer's, trained with it (not decayed either).  The
    optimizer holds the weights of `inputs` and the `grads` that the trainer was built with: change
    them in place; step() refuses others."""

    def __init__(self, inputs, capacity, device="cuda", fill_order="token", overflow="drop", tiled=False,
                 shared_tiled=False, alpha=0.01, z_coeff=0.001, seq_offsets=None, token_mask=None, weight_decay=0.01,
                 norm_weight=None, norm_eps=1e-6, **adamw):
        w = inputs.workload
        self.layer = MoELayer(inputs, capacity, device, fill_order, overflow, tiled, shared_tiled,
                              norm_weight=norm_weight, norm_eps=norm_eps)
        desc = self.layer.desc
        if desc.dtype != MOE_DTYPE_BF16:
            raise ValueError("training is implemented for bf16 layers")
        T, E, S = w.num_tokens, w.num_experts, _num_seqs(seq_offsets)
        self.alpha, self.z_coeff, self.seq_offsets, self.token_mask = alpha, z_coeff, seq_offsets, token_mask
        f32 = dict(dtype=torch.float32, device=device)
        i32 = dict(dtype=torch.int32, device=device)
        self.counts, self.seq_tokens = torch.zeros((S, E), **i32), torch.zeros((S,), **i32)
        self.mean_probs, self.losses = torch.zeros((S, E), **f32), torch.zeros((2,), **f32)
        self.dlogits = torch.zeros((T, E), **f32)
        self.dx = torch.zeros_like(inputs.x)
        names = ["router", "gate_up", "down"] + (["shared_gate_up", "shared_down"] if w.d_ff_shared else [])
        weights = [getattr(inputs, "w_" + n) for n in names]
        self.grads = {"dw_" + n: torch.zeros(p.shape, dtype=torch.float32 if n == "router" else p.dtype, device=device)
                      for n, p in zip(names, weights)}
        self.balance_ws = workspace(moe_balance_workspace_size(desc, S), device)
        self.backward_ws = workspace(moe_backward_workspace_size(desc), device)
        if not isinstance(weight_decay, (list, tuple)):
            weight_decay = [0.0] + [weight_decay] * (len(names) - 1) + [0.0] * (norm_weight is not None)
        if norm_weight is not None:
            self.grads["dw_norm"] = torch.zeros((w.d_model,), **f32)
            self.norm_ws = workspace(moe_rms_norm_backward_workspace_size(T, w.d_model), device)
            names, weights = names + ["norm"], weights + [norm_weight]
        self._names = names
        self.optimizer = MoEAdamW(weights, [self.grads["dw_" + n] for n in names], weight_decay=weight_decay, **adamw)

    def forward(self, residual=None):
        return self.layer.forward(with_routing=True, residual=residual)

    def backward(self, dy, dh=None):
        """Gradients of sum(dy * out) + losses[0] + losses[1] of the last forward; returns dx.  With a norm dx is the
        gradient of inputs.x and of the residual; dh, the gradient that reaches the layer's h, adds to it."""
        i, r, desc = self.layer.inputs, self.layer.routing, self.layer.desc
        norm = self.layer.norm_weight
        if dh is not None and norm is None:
            raise ValueError("dh is a gradient on the norm's h: construct MoETrainer with norm_weight")
        x = i.x if norm is None else self.layer.normed
        moe_balance_loss(desc, r["logits"], r["topk_ids"], self.alpha, self.z_coeff, self.counts, self.seq_tokens,
                         self.mean_probs, self.losses, self.balance_ws, token_mask=self.token_mask,
                         seq_offsets=self.seq_offsets, dlogits=self.dlogits)
        moe_backward(desc, i.w_router, i.w_gate_up, i.w_down, x, r, dy, self.dx, self.grads, self.backward_ws,
                     w_shared_gate_up=i.w_shared_gate_up, w_shared_down=i.w_shared_down, tiled=self.layer.tiled,
                     shared_tiled=self.layer.shared_tiled, dlogits=self.dlogits)
        if norm is not None:
            moe_rms_norm_backward(self.dx, self.layer.h, norm, self.layer.rstd, self.dx, self.grads["dw_norm"],
                                  self.norm_ws, dh=dh)
        return self.dx

    def step(self) -> None:
        for n, p, g in zip(self._names, self.optimizer.params, self.optimizer.grads):
            now = self.layer.norm_weight if n == "norm" else getattr(self.layer.inputs, "w_" + n)
            if now.data_ptr() != p.data_ptr():
                raise RuntimeError(f"{'norm_weight' if n == 'norm' else 'inputs.w_' + n} is not the tensor that the "
                                   "optimizer updates: build the trainer again")
            if self.grads["dw_" + n].data_ptr() != g.data_ptr():
                raise RuntimeError(f"grads['dw_{n}'] is not the tensor that the optimizer reads: build the trainer again")
        self.optimizer.step()
        i, L = self.layer.inputs, self.layer
        if L.tiled is not None:
            moe_tile_expert_weights(L.desc, i.w_gate_up.shape[0], i.w_gate_up, i.w_down, *L.tiled)
        if L.shared_tiled is not None:
            tile_shared_weights(L.desc, i.w_shared_gate_up, i.w_shared_down, *L.shared_tiled)

    def train_step(self, dy, residual=None, dh=None):
        """forward(residual), backward(dy, dh), step; returns the forward's out."""
        out = self.forward(residual)
        self.backward(dy, dh)
        self.step()
        return out
