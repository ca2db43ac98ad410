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
    "moe_adamw_read_states",
]
MOE_MAX_SEQS = 65536
MOE_ADAMW_BLOCK = 256
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
    if t.dtype is not dtypes and not (isinstance(dtypes, tuple) and t.dtype in dtypes):
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtypes}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.get_device() != (_device() if dev is None else dev):
        raise ValueError(f"{name} is on {t.device}; the library runs on the current GPU")
    return t.data_ptr()


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


class MoELayer:
    """Holds one layer's device tensors and a workspace, and runs moe_forward.

    Convenience only: allocation happens here, once, never inside a forward call."""

    def __init__(self, inputs, capacity, device="cuda", fill_order="token", overflow="drop", tiled=False,
                 shared_tiled=False):
        w = inputs.workload
        self.inputs = inputs
        self.desc = make_desc(w.num_tokens, w.d_model, w.d_ff, w.num_experts, w.top_k, capacity,
                              w.d_ff_shared, w.torch_dtype, fill_order=fill_order, overflow=overflow)
        self.ws = workspace(moe_workspace_size(self.desc), device)
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

    def forward_staged(self, events, with_routing=False, stream=None):
        i = self.inputs
        moe_forward_staged(self.desc, i.w_router, i.w_gate_up, i.w_down, i.x, i.logit_offset, self.out, self.ws,
                           events, routing=self.routing if with_routing else None,
                           w_shared_gate_up=i.w_shared_gate_up, w_shared_down=i.w_shared_down, stream=stream,
                           tiled=self.tiled, shared_tiled=self.shared_tiled)
        return self.out

    def forward(self, with_routing=True, stream=None):
        i = self.inputs
        moe_forward(self.desc, i.w_router, i.w_gate_up, i.w_down, i.x, i.logit_offset, self.out, self.ws,
                    routing=self.routing if with_routing else None, w_shared_gate_up=i.w_shared_gate_up,
                    w_shared_down=i.w_shared_down, stream=stream, tiled=self.tiled, shared_tiled=self.shared_tiled)
        return self.out


class MoETrainer:
    """One bf16 layer's training step: moe_forward, the balance and z losses with their gradient
    (moe_balance_loss), moe_backward_with_dlogits, the clipped AdamW step, and the tile-major copies
    rewritten from the new weights.

    Buffers are allocated here, once; the optimizer's options (lr, weight_decay, max_grad_norm,
    state_bits, master_weights, capturable, ...) are MoEAdamW's.  The router is not decayed unless
    weight_decay is given per tensor (router, gate_up, down[, shared gate_up, shared down]).  The
    optimizer holds the weights of `inputs` and the `grads` that the trainer was built with: change
    them in place; step() refuses others."""

    def __init__(self, inputs, capacity, device="cuda", fill_order="token", overflow="drop", tiled=False,
                 shared_tiled=False, alpha=0.01, z_coeff=0.001, seq_offsets=None, token_mask=None, weight_decay=0.01,
                 **adamw):
        w = inputs.workload
        self.layer = MoELayer(inputs, capacity, device, fill_order, overflow, tiled, shared_tiled)
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
            weight_decay = [0.0] + [weight_decay] * (len(names) - 1)
        self._names = names
        self.optimizer = MoEAdamW(weights, [self.grads["dw_" + n] for n in names], weight_decay=weight_decay, **adamw)

    def forward(self):
        return self.layer.forward(with_routing=True)

    def backward(self, dy):
        """Gradients of sum(dy * out) + losses[0] + losses[1] of the last forward; returns dx."""
        i, r, desc = self.layer.inputs, self.layer.routing, self.layer.desc
        moe_balance_loss(desc, r["logits"], r["topk_ids"], self.alpha, self.z_coeff, self.counts, self.seq_tokens,
                         self.mean_probs, self.losses, self.balance_ws, token_mask=self.token_mask,
                         seq_offsets=self.seq_offsets, dlogits=self.dlogits)
        moe_backward(desc, i.w_router, i.w_gate_up, i.w_down, i.x, r, dy, self.dx, self.grads, self.backward_ws,
                     w_shared_gate_up=i.w_shared_gate_up, w_shared_down=i.w_shared_down, tiled=self.layer.tiled,
                     shared_tiled=self.layer.shared_tiled, dlogits=self.dlogits)
        return self.dx

    def step(self) -> None:
        for n, p, g in zip(self._names, self.optimizer.params, self.optimizer.grads):
            if getattr(self.layer.inputs, "w_" + n).data_ptr() != p.data_ptr():
                raise RuntimeError(f"inputs.w_{n} is not the tensor that the optimizer updates: build the trainer again")
            if self.grads["dw_" + n].data_ptr() != g.data_ptr():
                raise RuntimeError(f"grads['dw_{n}'] is not the tensor that the optimizer reads: build the trainer again")
        self.optimizer.step()
        i, L = self.layer.inputs, self.layer
        if L.tiled is not None:
            moe_tile_expert_weights(L.desc, i.w_gate_up.shape[0], i.w_gate_up, i.w_down, *L.tiled)
        if L.shared_tiled is not None:
            tile_shared_weights(L.desc, i.w_shared_gate_up, i.w_shared_down, *L.shared_tiled)

    def train_step(self, dy):
        """forward, backward(dy), step; returns the forward's out."""
        out = self.forward()
        self.backward(dy)
        self.step()
        return out
