"""Thin ctypes binding of libep (include/ep.h): argument marshalling only.

Every function below has the name of the C entry point it calls and takes
torch tensors that already live on the GPU; it checks dtype / shape /
contiguity, passes raw pointers and the current CUDA stream, and raises
EPError on a non-zero return code.  Every step of the path runs in libep's
CUDA kernels: there is no CPU or PyTorch fallback, and importing this
module on a machine without the built library raises.

The alloc_* helpers only create output tensors of the documented shapes
(torch is the memory owner); they do no compute.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

from . import _build

EP_OK = 0
EP_ERR_INVALID_ARG = 1
EP_ERR_CAPACITY = 2
EP_ERR_TIMEOUT = 3
EP_ERR_CUDA = 4
EP_ERR_STATE = 5
EP_ERR_TOO_LARGE = 6

EP_FP8_NONE = 0
EP_FP8_E4M3_F32_SCALE = 1
EP_FP8_E4M3_UE8M0 = 2

EXPORTS = (
    "ep_workspace_size", "ep_get_dispatch_layout", "ep_notify_dispatch", "ep_dispatch",
    "ep_combine", "ep_ll_dispatch", "ep_ll_combine", "ep_clean_ll_buffer", "ep_read_status",
    "ep_host_wait_counters", "ep_launch_count", "ep_error_string", "ep_rank_ids",
    "ep_rank_recv_topk", "ep_rank_combine", "ep_set_num_sms", "ep_get_num_sms",
    "ep_format_e4m3", "ep_format_bf16", "ep_layout_notify", "ep_layout_notify_dispatch",
    "ep_gate_topk", "ep_gate_topk_backward", "ep_expert_glu", "ep_expert_glu_backward",
    "ep_expert_linear", "ep_expert_linear_backward", "ep_moe_few_workspace_size", "ep_moe_few",
    "ep_orthogonalize_workspace_size", "ep_orthogonalize", "ep_muon_update",
)

EP_MOE_FEW_TOKENS = 64

EP_DTYPE_F32 = 0
EP_DTYPE_BF16 = 1

EP_GATE_SOFTMAX = 0
EP_GATE_SOFTMAX_TOPK = 1
GATE_SCORES = {"softmax": EP_GATE_SOFTMAX, "softmax_topk": EP_GATE_SOFTMAX_TOPK}

EP_ACT_NONE = 0
EP_ACT_RELU = 1
EP_ACT_SILU = 2
EP_ACT_GELU = 3
ACTS = {"none": EP_ACT_NONE, "relu": EP_ACT_RELU, "silu": EP_ACT_SILU, "gelu": EP_ACT_GELU}


class EPError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {error_string(code)} (code {code})")


_lib = None
_P, _I, _I64, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
_F = ctypes.c_float


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libep.so (building it with nvcc first if it is missing/stale)."""
    global _lib
    if _lib is not None:
        return _lib
    if build_if_missing:
        _build.build()
    if not os.path.exists(_build.LIB):
        raise RuntimeError(f"libep.so not found at {_build.LIB}; build it with __graft_entry__.build()")
    L = ctypes.CDLL(_build.LIB)
    L.ep_workspace_size.argtypes = [_I, _I, _I, _I, _I]
    L.ep_workspace_size.restype = _SZ
    L.ep_get_dispatch_layout.argtypes = [_P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _SZ, _P, _P]
    L.ep_notify_dispatch.argtypes = [_P, _P, _I, _I, _I, _I64, _P, _P, _P, _P, _P, _I, _P, _P]
    L.ep_dispatch.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I64, _P, _P, _P, _P,
                              _P, _SZ, _P, _P]
    L.ep_combine.argtypes = [_P, _P, _P, _I, _I, _I, _I, _I64, _P, _P, _P]
    L.ep_ll_dispatch.argtypes = [_P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P,
                                 _SZ, _P, _P]
    L.ep_ll_combine.argtypes = [_P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P]
    L.ep_clean_ll_buffer.argtypes = [_P, _I, _I, _P, _SZ, _P]
    L.ep_rank_ids.argtypes = [_P, _I, _I, _I, _I, _P, _P, _P]
    L.ep_rank_recv_topk.argtypes = [_P, _P, _P, _I, _I, _I, _I, _I64, _P, _P, _P, _P]
    L.ep_rank_combine.argtypes = [_P, _P, _I, _I, _I, _I, _I64, _P, _P, _P]
    L.ep_read_status.argtypes = [_P, _P, _P]
    L.ep_host_wait_counters.argtypes = [_P, _I, _I]
    L.ep_layout_notify.argtypes = [_P, _I, _I, _I, _I, _I, _I64, _P, _P, _P, _P, _P, _P, _P, _P,
                                   _P, _I, _P, _SZ, _P, _P]
    L.ep_layout_notify.restype = _I
    L.ep_layout_notify_dispatch.argtypes = [_P, _P, _I, _I, _I, _I, _I, _I, _I, _I64, _I64, _P, _P,
                                            _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P,
                                            _P]
    L.ep_layout_notify_dispatch.restype = _I
    L.ep_format_e4m3.argtypes = [_P, _P, _I64, _P]
    L.ep_format_e4m3.restype = _I
    L.ep_format_bf16.argtypes = [_P, _P, _I64, _P]
    L.ep_format_bf16.restype = _I
    L.ep_gate_topk.argtypes = [_P, _I, _I, _I, _I, _I, _I, _P, _P, _P]
    L.ep_gate_topk_backward.argtypes = [_P, _I, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P]
    L.ep_expert_glu.argtypes = [_P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I64, _I, _P, _P, _P,
                                _P, _P]
    L.ep_expert_glu_backward.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I64, _I, _P, _P,
                                         _P, _P, _P]
    L.ep_expert_linear.argtypes = [_P, _P, _P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I64, _I,
                                   _P, _P, _P, _P]
    L.ep_expert_linear_backward.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I64, _I, _P,
                                            _P, _P, _P, _P, _P]
    L.ep_moe_few_workspace_size.argtypes = [_I, _I, _I, _I, _I]
    L.ep_moe_few_workspace_size.restype = _SZ
    L.ep_moe_few.argtypes = [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P,
                             _SZ, _P, _P]
    L.ep_orthogonalize_workspace_size.argtypes = [_I, _I, _I]
    L.ep_orthogonalize_workspace_size.restype = _SZ
    L.ep_orthogonalize.argtypes = [_P, _I, _I, _I, _I, _I, _P, _F, _P, _P, _SZ, _P, _P]
    L.ep_muon_update.argtypes = [_P, _I, _P, _P, _P, _I, _I, _I, _F, _F, _F, _I, _F, _I, _P, _F,
                                 _P, _SZ, _P, _P]
    L.ep_set_num_sms.argtypes = [_I]
    L.ep_set_num_sms.restype = _I
    L.ep_get_num_sms.argtypes = []
    L.ep_get_num_sms.restype = _I
    L.ep_launch_count.argtypes = []
    L.ep_launch_count.restype = ctypes.c_uint64
    L.ep_error_string.argtypes = [_I]
    L.ep_error_string.restype = ctypes.c_char_p
    for name in ("ep_get_dispatch_layout", "ep_notify_dispatch", "ep_dispatch", "ep_combine",
                 "ep_ll_dispatch", "ep_ll_combine", "ep_clean_ll_buffer", "ep_read_status",
                 "ep_host_wait_counters", "ep_rank_ids", "ep_rank_recv_topk", "ep_rank_combine",
                 "ep_gate_topk", "ep_gate_topk_backward", "ep_expert_glu",
                 "ep_expert_glu_backward", "ep_expert_linear", "ep_expert_linear_backward",
                 "ep_moe_few", "ep_orthogonalize", "ep_muon_update"):
        getattr(L, name).restype = _I
    _lib = L
    return L


def error_string(code: int) -> str:
    return load().ep_error_string(int(code)).decode()


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    # the raw handle of torch.cuda.current_stream(), without the object (2.8 us of a call's host time)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _need(t: torch.Tensor | None, dtype, shape=None, name="tensor", optional=False):
    if (t is not None and t.is_cuda and (dtype is None or t.dtype == dtype) and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        return
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _here(*tensors):
    """The tensors are on the current device, whose stream the call uses."""
    dev = torch._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensor on device {t.get_device()}, the current one is {dev}")


def _need_out(t: torch.Tensor, dtype, shape, name="out"):
    """A combine's output: a CUDA tensor, or a pinned host tensor that the
    kernel writes across the host link."""
    if not t.is_cuda and not t.is_pinned():
        raise ValueError(f"{name} must be a CUDA tensor or pinned host memory")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _check(rc: int, where: str):
    if rc != EP_OK:
        raise EPError(rc, where)


def _scale_dtype(fp8_mode: int):
    return torch.float32 if fp8_mode == EP_FP8_E4M3_F32_SCALE else torch.uint8


# ------------------------------------------------------------------ entry points

def ep_workspace_size(R: int, T_r: int, k: int, E: int, H: int) -> int:
    return int(load().ep_workspace_size(R, T_r, k, E, H))


def ep_get_dispatch_layout(topk_idx, num_experts, num_tokens_per_rank, num_tokens_per_expert,
                           is_token_in_rank, slot_rank, workspace, status=None, stream=None):
    R, T_r, k = topk_idx.shape
    E = num_experts
    _need(topk_idx, torch.int64, name="topk_idx")
    _need(num_tokens_per_rank, torch.int32, (R, R), "num_tokens_per_rank")
    _need(num_tokens_per_expert, torch.int32, (R, E), "num_tokens_per_expert")
    _need(is_token_in_rank, torch.uint8, (R, T_r, R), "is_token_in_rank")
    _need(slot_rank, torch.int32, (R, T_r, k), "slot_rank")
    _need(workspace, torch.uint8, name="workspace")
    _need(status, torch.int32, (1,), "status", optional=True)
    rc = load().ep_get_dispatch_layout(_ptr(topk_idx), R, T_r, k, E, _ptr(num_tokens_per_rank),
                                       _ptr(num_tokens_per_expert), _ptr(is_token_in_rank),
                                       _ptr(slot_rank), _ptr(workspace), workspace.numel(),
                                       _ptr(status), _stream(stream))
    _check(rc, "ep_get_dispatch_layout")


def ep_notify_dispatch(num_tokens_per_rank, num_tokens_per_expert, expert_alignment,
                       num_worst_tokens, rank_prefix_matrix, expert_prefix,
                       num_recv_tokens_per_expert, psum, host_recv_rows=None, timeout_ms=10000,
                       status=None, stream=None):
    R, E = num_tokens_per_expert.shape
    E_l = E // R
    _need(num_tokens_per_rank, torch.int32, (R, R), "num_tokens_per_rank")
    _need(num_tokens_per_expert, torch.int32, (R, E), "num_tokens_per_expert")
    _need(rank_prefix_matrix, torch.int32, (R, R), "rank_prefix_matrix")
    _need(expert_prefix, torch.int32, (R + 1, E), "expert_prefix")
    _need(num_recv_tokens_per_expert, torch.int32, (R, E_l), "num_recv_tokens_per_expert")
    _need(psum, torch.int64, (R, E_l + 1), "psum")
    _need(status, torch.int32, (1,), "status", optional=True)
    if host_recv_rows is not None:
        if host_recv_rows.is_cuda or not host_recv_rows.is_pinned() or \
                host_recv_rows.dtype != torch.int64 or host_recv_rows.numel() < R:
            raise ValueError("host_recv_rows must be a pinned host int64 tensor of >= R entries")
    rc = load().ep_notify_dispatch(_ptr(num_tokens_per_rank), _ptr(num_tokens_per_expert), R, E,
                                   expert_alignment, num_worst_tokens, _ptr(rank_prefix_matrix),
                                   _ptr(expert_prefix), _ptr(num_recv_tokens_per_expert),
                                   _ptr(psum), _ptr(host_recv_rows), timeout_ms, _ptr(status),
                                   _stream(stream))
    _check(rc, "ep_notify_dispatch")


def ep_layout_notify(topk_idx, num_experts, expert_alignment, num_worst_tokens, lay, nt,
                     workspace, host_recv_rows=None, timeout_ms=10000, status=None, stream=None):
    """ep_get_dispatch_layout + ep_notify_dispatch in one launch; `lay` and
    `nt` are the dicts of alloc_layout / alloc_notify."""
    R, T_r, k = topk_idx.shape
    E = num_experts
    E_l = E // R
    _need(topk_idx, torch.int64, name="topk_idx")
    _need(lay["num_tokens_per_rank"], torch.int32, (R, R), "num_tokens_per_rank")
    _need(lay["num_tokens_per_expert"], torch.int32, (R, E), "num_tokens_per_expert")
    _need(lay["is_token_in_rank"], torch.uint8, (R, T_r, R), "is_token_in_rank")
    _need(lay["slot_rank"], torch.int32, (R, T_r, k), "slot_rank")
    _need(nt["rank_prefix_matrix"], torch.int32, (R, R), "rank_prefix_matrix")
    _need(nt["expert_prefix"], torch.int32, (R + 1, E), "expert_prefix")
    _need(nt["num_recv_tokens_per_expert"], torch.int32, (R, E_l), "num_recv_tokens_per_expert")
    _need(nt["psum"], torch.int64, (R, E_l + 1), "psum")
    _need(workspace, torch.uint8, name="workspace")
    _need(status, torch.int32, (1,), "status", optional=True)
    if host_recv_rows is not None:
        if host_recv_rows.is_cuda or not host_recv_rows.is_pinned() or \
                host_recv_rows.dtype != torch.int64 or host_recv_rows.numel() < R:
            raise ValueError("host_recv_rows must be a pinned host int64 tensor of >= R entries")
    rc = load().ep_layout_notify(_ptr(topk_idx), R, T_r, k, E, expert_alignment, num_worst_tokens,
                                 _ptr(lay["num_tokens_per_rank"]), _ptr(lay["num_tokens_per_expert"]),
                                 _ptr(lay["is_token_in_rank"]), _ptr(lay["slot_rank"]),
                                 _ptr(nt["rank_prefix_matrix"]), _ptr(nt["expert_prefix"]),
                                 _ptr(nt["num_recv_tokens_per_expert"]), _ptr(nt["psum"]),
                                 _ptr(host_recv_rows), timeout_ms, _ptr(workspace),
                                 workspace.numel(), _ptr(status), _stream(stream))
    _check(rc, "ep_layout_notify")


def ep_layout_notify_dispatch(x, topk_idx, num_experts, fp8_mode, expert_alignment,
                              num_worst_tokens, cap_rows, lay, nt, d, workspace, status=None,
                              stream=None):
    """Fixed-shape normal mode in one call: layout + notify (one launch),
    then the dispatch as its programmatic dependent.  `lay`, `nt`, `d` are
    the dicts of alloc_layout / alloc_notify / alloc_dispatch."""
    R, T_r, H = x.shape
    k = topk_idx.shape[2]
    E = num_experts
    E_l = E // R
    _need(x, torch.bfloat16, (R, T_r, H), "x")
    _need(topk_idx, torch.int64, (R, T_r, k), "topk_idx")
    for key, dt, shape in (("num_tokens_per_rank", torch.int32, (R, R)),
                           ("num_tokens_per_expert", torch.int32, (R, E)),
                           ("is_token_in_rank", torch.uint8, (R, T_r, R)),
                           ("slot_rank", torch.int32, (R, T_r, k))):
        _need(lay[key], dt, shape, key)
    for key, dt, shape in (("rank_prefix_matrix", torch.int32, (R, R)),
                           ("expert_prefix", torch.int32, (R + 1, E)),
                           ("num_recv_tokens_per_expert", torch.int32, (R, E_l)),
                           ("psum", torch.int64, (R, E_l + 1))):
        _need(nt[key], dt, shape, key)
    rdt = torch.bfloat16 if fp8_mode == EP_FP8_NONE else torch.uint8
    _need(d["recv_x"], rdt, (R, cap_rows, H), "recv_x")
    if fp8_mode != EP_FP8_NONE:
        _need(d["recv_scales"], _scale_dtype(fp8_mode), (R, H // 128, cap_rows), "recv_scales")
    _need(d["recv_src_idx"], torch.int32, (R, cap_rows), "recv_src_idx")
    _need(d["combine_idx"], torch.int32, (R, T_r, k), "combine_idx")
    _need(workspace, torch.uint8, name="workspace")
    _need(status, torch.int32, (1,), "status", optional=True)
    rc = load().ep_layout_notify_dispatch(
        _ptr(x), _ptr(topk_idx), R, T_r, H, E, k, fp8_mode, expert_alignment, num_worst_tokens,
        cap_rows, _ptr(lay["num_tokens_per_rank"]), _ptr(lay["num_tokens_per_expert"]),
        _ptr(lay["is_token_in_rank"]), _ptr(lay["slot_rank"]), _ptr(nt["rank_prefix_matrix"]),
        _ptr(nt["expert_prefix"]), _ptr(nt["num_recv_tokens_per_expert"]), _ptr(nt["psum"]),
        _ptr(d["recv_x"]), _ptr(d["recv_scales"]) if fp8_mode != EP_FP8_NONE else None,
        _ptr(d["recv_src_idx"]), _ptr(d["combine_idx"]), _ptr(workspace), workspace.numel(),
        _ptr(status), _stream(stream))
    _check(rc, "ep_layout_notify_dispatch")


def ep_dispatch(x, topk_idx, slot_rank, expert_prefix, psum, num_experts, fp8_mode, cap_rows,
                recv_x, recv_scales, recv_src_idx, combine_idx, workspace=None, status=None,
                stream=None):
    R, T_r, H = x.shape
    k = topk_idx.shape[2]
    E = num_experts
    E_l = E // R
    _need(x, torch.bfloat16, (R, T_r, H), "x")
    _need(topk_idx, torch.int64, (R, T_r, k), "topk_idx")
    _need(slot_rank, torch.int32, (R, T_r, k), "slot_rank")
    _need(expert_prefix, torch.int32, (R + 1, E), "expert_prefix")
    _need(psum, torch.int64, (R, E_l + 1), "psum")
    rdt = torch.bfloat16 if fp8_mode == EP_FP8_NONE else torch.uint8
    _need(recv_x, rdt, (R, cap_rows, H), "recv_x")
    if fp8_mode != EP_FP8_NONE:
        _need(recv_scales, _scale_dtype(fp8_mode), (R, H // 128, cap_rows), "recv_scales")
    _need(recv_src_idx, torch.int32, (R, cap_rows), "recv_src_idx")
    _need(combine_idx, torch.int32, (R, T_r, k), "combine_idx")
    _need(workspace, torch.uint8, name="workspace", optional=fp8_mode == EP_FP8_NONE)
    _need(status, torch.int32, (1,), "status", optional=True)
    rc = load().ep_dispatch(_ptr(x), _ptr(topk_idx), _ptr(slot_rank), _ptr(expert_prefix),
                            _ptr(psum), R, T_r, H, E, k, fp8_mode, cap_rows, _ptr(recv_x),
                            _ptr(recv_scales) if fp8_mode != EP_FP8_NONE else None,
                            _ptr(recv_src_idx), _ptr(combine_idx), _ptr(workspace),
                            0 if workspace is None else workspace.numel(), _ptr(status),
                            _stream(stream))
    _check(rc, "ep_dispatch")


def ep_combine(y, topk_weights, combine_idx, cap_rows, out, status=None, stream=None):
    R, T_r, k = combine_idx.shape
    H = out.shape[2]
    _need(y, torch.bfloat16, (R, cap_rows, H), "y")
    _need(topk_weights, torch.float32, (R, T_r, k), "topk_weights")
    _need(combine_idx, torch.int32, (R, T_r, k), "combine_idx")
    _need_out(out, torch.bfloat16, (R, T_r, H))
    _need(status, torch.int32, (1,), "status", optional=True)
    rc = load().ep_combine(_ptr(y), _ptr(topk_weights), _ptr(combine_idx), R, T_r, H, k, cap_rows,
                           _ptr(out), _ptr(status), _stream(stream))
    _check(rc, "ep_combine")


def ep_ll_dispatch(x, topk_idx, num_experts, max_tokens_per_rank, fp8_mode, packed_recv_x,
                   packed_recv_scales, packed_recv_src_info, layout_range, recv_count, combine_idx,
                   workspace, status=None, stream=None):
    R, T_r, H = x.shape
    k = topk_idx.shape[2]
    E = num_experts
    E_l = E // R
    S = R * max_tokens_per_rank
    _need(x, torch.bfloat16, (R, T_r, H), "x")
    _need(topk_idx, torch.int64, (R, T_r, k), "topk_idx")
    rdt = torch.bfloat16 if fp8_mode == EP_FP8_NONE else torch.uint8
    _need(packed_recv_x, rdt, (R, E_l, S, H), "packed_recv_x")
    if fp8_mode != EP_FP8_NONE:
        _need(packed_recv_scales, _scale_dtype(fp8_mode), (R, E_l, H // 128, S),
              "packed_recv_scales")
    _need(packed_recv_src_info, torch.int32, (R, E_l, S), "packed_recv_src_info")
    _need(layout_range, torch.int64, (R, E_l, R), "layout_range")
    _need(recv_count, torch.int32, (R, E_l), "recv_count")
    _need(combine_idx, torch.int32, (R, T_r, k), "combine_idx")
    _need(workspace, torch.uint8, name="workspace")
    _need(status, torch.int32, (1,), "status", optional=True)
    rc = load().ep_ll_dispatch(_ptr(x), _ptr(topk_idx), R, T_r, H, E, k, max_tokens_per_rank,
                               fp8_mode, _ptr(packed_recv_x),
                               _ptr(packed_recv_scales) if fp8_mode != EP_FP8_NONE else None,
                               _ptr(packed_recv_src_info), _ptr(layout_range), _ptr(recv_count),
                               _ptr(combine_idx), _ptr(workspace), workspace.numel(),
                               _ptr(status), _stream(stream))
    _check(rc, "ep_ll_dispatch")


def ep_ll_combine(y, topk_weights, combine_idx, num_experts, max_tokens_per_rank, out,
                  status=None, stream=None):
    R, T_r, k = combine_idx.shape
    H = out.shape[2]
    E = num_experts
    E_l = E // R
    _need(y, torch.bfloat16, (R, E_l, R * max_tokens_per_rank, H), "y")
    _need(topk_weights, torch.float32, (R, T_r, k), "topk_weights")
    _need(combine_idx, torch.int32, (R, T_r, k), "combine_idx")
    _need_out(out, torch.bfloat16, (R, T_r, H))
    _need(status, torch.int32, (1,), "status", optional=True)
    rc = load().ep_ll_combine(_ptr(y), _ptr(topk_weights), _ptr(combine_idx), R, T_r, H, E, k,
                              max_tokens_per_rank, _ptr(out), _ptr(status), _stream(stream))
    _check(rc, "ep_ll_combine")


def ep_clean_ll_buffer(recv_count, num_ranks, num_experts, workspace, stream=None):
    _need(recv_count, torch.int32, name="recv_count", optional=True)
    _need(workspace, torch.uint8, name="workspace", optional=True)
    rc = load().ep_clean_ll_buffer(_ptr(recv_count), num_ranks, num_experts, _ptr(workspace),
                                   0 if workspace is None else workspace.numel(), _stream(stream))
    _check(rc, "ep_clean_ll_buffer")


def ep_rank_ids(topk_idx, num_experts, rank_ids, status=None, stream=None):
    R, T_r, k = topk_idx.shape
    _need(topk_idx, torch.int64, name="topk_idx")
    _need(rank_ids, torch.int64, (R, T_r, k), "rank_ids")
    _need(status, torch.int32, (1,), "status", optional=True)
    rc = load().ep_rank_ids(_ptr(topk_idx), R, T_r, k, num_experts, _ptr(rank_ids), _ptr(status),
                            _stream(stream))
    _check(rc, "ep_rank_ids")


def ep_rank_recv_topk(topk_idx, topk_weights, combine_idx, num_experts, cap_rows, recv_topk_idx,
                      recv_topk_weights, status=None, stream=None):
    R, T_r, k = topk_idx.shape
    _need(topk_idx, torch.int64, name="topk_idx")
    _need(topk_weights, torch.float32, (R, T_r, k), "topk_weights")
    _need(combine_idx, torch.int32, (R, T_r, k), "combine_idx")
    _need(recv_topk_idx, torch.int64, (R, cap_rows, k), "recv_topk_idx")
    _need(recv_topk_weights, torch.float32, (R, cap_rows, k), "recv_topk_weights")
    _need(status, torch.int32, (1,), "status", optional=True)
    rc = load().ep_rank_recv_topk(_ptr(topk_idx), _ptr(topk_weights), _ptr(combine_idx), R, T_r,
                                  k, num_experts, cap_rows, _ptr(recv_topk_idx),
                                  _ptr(recv_topk_weights), _ptr(status), _stream(stream))
    _check(rc, "ep_rank_recv_topk")


def ep_rank_combine(y, combine_idx, cap_rows, out, status=None, stream=None):
    R, T_r, k = combine_idx.shape
    H = out.shape[2]
    _need(y, torch.bfloat16, (R, cap_rows, H), "y")
    _need(combine_idx, torch.int32, (R, T_r, k), "combine_idx")
    _need_out(out, torch.bfloat16, (R, T_r, H))
    _need(status, torch.int32, (1,), "status", optional=True)
    rc = load().ep_rank_combine(_ptr(y), _ptr(combine_idx), R, T_r, H, k, cap_rows, _ptr(out),
                                _ptr(status), _stream(stream))
    _check(rc, "ep_rank_combine")


def _gate_dtype(logits):
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"logits: dtype {logits.dtype}, expected float32 or bfloat16")
    return EP_DTYPE_F32 if logits.dtype == torch.float32 else EP_DTYPE_BF16


def ep_gate_topk(logits, score, topk_idx, topk_weights, stream=None):
    """Router top-k: logits [R, T_r, E] -> topk_idx, topk_weights [R, T_r, k]."""
    R, T_r, E = logits.shape
    k = topk_idx.shape[2]
    dtype = _gate_dtype(logits)
    _need(logits, None, name="logits")
    _need(topk_idx, torch.int64, (R, T_r, k), "topk_idx")
    _need(topk_weights, torch.float32, (R, T_r, k), "topk_weights")
    rc = load().ep_gate_topk(_ptr(logits), dtype, R, T_r, E, k, score, _ptr(topk_idx),
                             _ptr(topk_weights), _stream(stream))
    _check(rc, "ep_gate_topk")


def ep_gate_topk_backward(logits, score, topk_idx, grad_topk_weights, grad_logits, status=None,
                          stream=None):
    """Gradient of ep_gate_topk's weights; ids outside [-1, E) count as unused,
    which only the status word says."""
    R, T_r, E = logits.shape
    k = topk_idx.shape[2]
    dtype = _gate_dtype(logits)
    _need(logits, None, name="logits")
    _need(topk_idx, torch.int64, (R, T_r, k), "topk_idx")
    _need(grad_topk_weights, torch.float32, (R, T_r, k), "grad_topk_weights")
    _need(grad_logits, logits.dtype, (R, T_r, E), "grad_logits")
    _need(status, torch.int32, (1,), "status", optional=True)
    rc = load().ep_gate_topk_backward(_ptr(logits), dtype, _ptr(topk_idx), _ptr(grad_topk_weights),
                                      R, T_r, E, k, score, _ptr(grad_logits), _ptr(status),
                                      _stream(stream))
    _check(rc, "ep_gate_topk_backward")


def _expert_rows(lead, E, counts, psum, status):
    """Checks the tables of a receive layout with leading dimensions `lead`
    ((R, cap_rows) with psum, (R, E_l, cap_rows) without); R and cap_rows."""
    R, cap = lead[0], lead[-1]
    if R == 0 or E % R != 0:
        raise ValueError(f"{E} experts on {R} ranks")
    if lead != ((R, cap) if psum is not None else (R, E // R, cap)):
        raise ValueError(f"rows: leading shape {tuple(lead)}, expected (R, cap_rows) with psum, "
                         "(R, E_l, cap_rows) without")
    _need(counts, torch.int32, name="counts")
    shape = counts.shape
    if shape != (R, E // R) and shape != (E,):
        raise ValueError(f"counts: shape {tuple(shape)}, expected {(E,)} or {(R, E // R)}")
    if psum is not None:
        _need(psum, torch.int64, (R, E // R + 1), "psum")
    if status is not None:
        _need(status, torch.int32, (1,), "status")
    return R, cap


def _expert_inputs(x, x_scales, w, w_scales, lead):
    """dtype and scale checks of the rows and weights; the FP8 mode."""
    if x_scales is None:
        _need(x, torch.bfloat16, name="x")
        _need(w, torch.bfloat16, name="w")
        if w_scales is not None:
            raise ValueError("w_scales without x_scales")
        return EP_FP8_NONE
    K = x.shape[-1]
    _need(x, torch.uint8, name="x")
    _need(w, torch.uint8, name="w")
    if x_scales.dtype == torch.float32:
        _need(x_scales, torch.float32, (*lead[:-1], K // 128, lead[-1]), "x_scales")
        _need(w_scales, None, name="w_scales")
        return EP_FP8_E4M3_F32_SCALE
    _need(x_scales, torch.uint8, (*lead[:-1], K // 128, lead[-1]), "x_scales")
    _need(w_scales, torch.uint8, (*w.shape[:-2], w.shape[-2] // 128, K // 128), "w_scales")
    return EP_FP8_E4M3_UE8M0


def ep_expert_glu(x, x_scales, w, w_scales, counts, psum, act, h, h_scales=None, gu=None,
                  status=None, stream=None):
    """h = act(x Wg^T) * (x Wu^T) over a receive layout; w [E, 2, I, H].

    x [R, cap_rows, H] with psum (normal layout), [R, E_l, cap_rows, H] without
    (packed).  bf16 (scales None), or E4M3 bytes with ue8m0 scales; with
    h_scales h is written as E4M3, with gu gate and up are kept in bf16.

    As in all the expert calls, rows past cap_rows are left out and a wait that
    ran out leaves outputs incomplete; only the status word says so
    (ep_read_status), and without one there is no sign."""
    *lead, H = x.shape
    lead = tuple(lead)
    E, two, I, Hw = w.shape
    if two != 2 or Hw != H:
        raise ValueError(f"w: shape {tuple(w.shape)}, expected (E, 2, I, {H})")
    R, cap = _expert_rows(lead, E, counts, psum, status)
    mode = _expert_inputs(x, x_scales, w, w_scales, lead)
    _need(h, torch.bfloat16 if h_scales is None else torch.uint8, (*lead, I), "h")
    if h_scales is not None:
        _need(h_scales, torch.uint8, (*lead[:-1], I // 128, cap), "h_scales")
    if gu is not None:
        _need(gu, torch.bfloat16, (*lead, 2, I), "gu")
    rc = load().ep_expert_glu(_ptr(x), _ptr(x_scales), _ptr(w), _ptr(w_scales), mode, _ptr(counts),
                              _ptr(psum), R, E, H, I, cap, act, _ptr(h), _ptr(h_scales), _ptr(gu),
                              _ptr(status), _stream(stream))
    _check(rc, "ep_expert_glu")


def ep_expert_glu_backward(dh, gu, x, w, counts, psum, act, dgu, dx, dw, status=None, stream=None):
    """Gradient of ep_expert_glu: dgu (gate and up), dx and dw (either may be
    None, and then w or x may be too).  Rows left out are told by status alone
    (see ep_expert_glu)."""
    lead, I = dh.shape[:-1], dh.shape[-1]
    some = w if w is not None else dw
    if some is None:
        raise ValueError("w or dw is required")
    E, H = some.shape[0], some.shape[-1]
    R, cap = _expert_rows(lead, E, counts, psum, status)
    _need(dh, torch.bfloat16, name="dh")
    _need(gu, torch.bfloat16, (*lead, 2, I), "gu")
    _need(dgu, torch.bfloat16, (*lead, 2, I), "dgu")
    _need(x, torch.bfloat16, (*lead, H), "x", optional=dw is None)
    _need(w, torch.bfloat16, (E, 2, I, H), "w", optional=dx is None)
    _need(dx, torch.bfloat16, (*lead, H), "dx", optional=True)
    _need(dw, torch.bfloat16, (E, 2, I, H), "dw", optional=True)
    rc = load().ep_expert_glu_backward(_ptr(dh), _ptr(gu), _ptr(x), _ptr(w), _ptr(counts),
                                       _ptr(psum), R, E, H, I, cap, act, _ptr(dgu), _ptr(dx),
                                       _ptr(dw), _ptr(status), _stream(stream))
    _check(rc, "ep_expert_glu_backward")


def ep_expert_linear(x, x_scales, w, w_scales, bias, residual, counts, psum, act, y, pre=None,
                     status=None, stream=None):
    """y = act(x W^T + bias) + residual over a receive layout; w [E, N, K].
    Rows left out are told by status alone (see ep_expert_glu)."""
    *lead, K = x.shape
    lead = tuple(lead)
    E, N, Kw = w.shape
    if Kw != K:
        raise ValueError(f"w: shape {tuple(w.shape)}, expected (E, N, {K})")
    R, cap = _expert_rows(lead, E, counts, psum, status)
    mode = _expert_inputs(x, x_scales, w, w_scales, lead)
    rows = (*lead, N)
    if bias is not None:
        _need(bias, torch.bfloat16, (E, N), "bias")
    if residual is not None:
        _need(residual, torch.bfloat16, rows, "residual")
    _need(y, torch.bfloat16, rows, "y")
    if pre is not None:
        _need(pre, torch.bfloat16, rows, "pre")
    rc = load().ep_expert_linear(_ptr(x), _ptr(x_scales), _ptr(w), _ptr(w_scales), mode, _ptr(bias),
                                 _ptr(residual), _ptr(counts), _ptr(psum), R, E, K, N, cap, act,
                                 _ptr(y), _ptr(pre), _ptr(status), _stream(stream))
    _check(rc, "ep_expert_linear")


def ep_expert_linear_backward(dy, pre, x, w, counts, psum, act, dpre, dx, dw, dbias=None,
                              status=None, stream=None):
    """Gradient of ep_expert_linear; pre and dpre are None without activation,
    dx, dw and dbias may each be None.  Rows left out are told by status alone
    (see ep_expert_glu)."""
    lead, N = dy.shape[:-1], dy.shape[-1]
    some = w if w is not None else dw
    if some is None:
        raise ValueError("w or dw is required")
    E, K = some.shape[0], some.shape[-1]
    R, cap = _expert_rows(lead, E, counts, psum, status)
    _need(dy, torch.bfloat16, name="dy")
    _need(pre, torch.bfloat16, (*lead, N), "pre", optional=act == EP_ACT_NONE)
    _need(dpre, torch.bfloat16, (*lead, N), "dpre", optional=act == EP_ACT_NONE)
    _need(x, torch.bfloat16, (*lead, K), "x", optional=dw is None)
    _need(w, torch.bfloat16, (E, N, K), "w", optional=dx is None)
    _need(dx, torch.bfloat16, (*lead, K), "dx", optional=True)
    _need(dw, torch.bfloat16, (E, N, K), "dw", optional=True)
    _need(dbias, torch.bfloat16, (E, N), "dbias", optional=True)
    rc = load().ep_expert_linear_backward(_ptr(dy), _ptr(pre), _ptr(x), _ptr(w), _ptr(counts),
                                          _ptr(psum), R, E, K, N, cap, act, _ptr(dpre), _ptr(dx),
                                          _ptr(dw), _ptr(dbias), _ptr(status), _stream(stream))
    _check(rc, "ep_expert_linear_backward")


def ep_moe_few_workspace_size(R: int, T_r: int, k: int, E: int, I: int) -> int:
    return int(load().ep_moe_few_workspace_size(R, T_r, k, E, I))


def ep_moe_few(x, topk_idx, topk_weights, w_gu, w_gu_scales, w_down, w_down_scales, act, out,
               workspace, status=None, stream=None):
    """A whole layer for at most EP_MOE_FEW_TOKENS tokens: out = sum over a
    token's slots of weight * W_down (act(W_gate x) * (W_up x)).

    x, out [R, T_r, H] bf16 (out may be x), topk_idx / topk_weights [R, T_r, k],
    w_gu [E, 2, I, H], w_down [E, H, I] in bf16 (scales None) or E4M3 bytes with
    ue8m0 scales of 128 x 128 blocks.  Ids outside [-1, E) count as unused, which
    only the status word says; workspace: alloc_moe_few_workspace."""
    R, T_r, H = x.shape
    k = topk_idx.shape[-1]
    E, two, I, Hw = w_gu.shape
    if two != 2 or Hw != H:
        raise ValueError(f"w_gu: shape {tuple(w_gu.shape)}, expected (E, 2, I, {H})")
    _need(x, torch.bfloat16, name="x")
    _need(topk_idx, torch.int64, (R, T_r, k), "topk_idx")
    _need(topk_weights, torch.float32, (R, T_r, k), "topk_weights")
    if w_gu_scales is None:
        mode, dtype = EP_FP8_NONE, torch.bfloat16
        if w_down_scales is not None:
            raise ValueError("w_down_scales without w_gu_scales")
    else:
        mode, dtype = EP_FP8_E4M3_UE8M0, torch.uint8
        _need(w_gu_scales, torch.uint8, (E, 2, I // 128, H // 128), "w_gu_scales")
        _need(w_down_scales, torch.uint8, (E, H // 128, I // 128), "w_down_scales")
    _need(w_gu, dtype, name="w_gu")
    _need(w_down, dtype, (E, H, I), "w_down")
    _need(out, torch.bfloat16, (R, T_r, H), "out")
    _need(workspace, torch.uint8, name="workspace")
    if status is not None:
        _need(status, torch.int32, (1,), "status")
    _here(x, topk_idx, topk_weights, w_gu, w_gu_scales, w_down, w_down_scales, out, workspace, status)
    rc = load().ep_moe_few(_ptr(x), _ptr(topk_idx), _ptr(topk_weights), _ptr(w_gu), _ptr(w_gu_scales),
                           _ptr(w_down), _ptr(w_down_scales), mode, R, T_r, k, E, H, I, act,
                           _ptr(out), _ptr(workspace), workspace.numel(), _ptr(status),
                           _stream(stream))
    _check(rc, "ep_moe_few")


def ep_orthogonalize_workspace_size(count: int, M: int, N: int) -> int:
    return int(load().ep_orthogonalize_workspace_size(count, M, N))


def _stack(g, steps):
    """(count, M, N), dtype and coefficients of a stack of matrices [..., M, N]."""
    if g.dim() < 2:
        raise ValueError(f"g: shape {tuple(g.shape)}, expected (..., M, N)")
    if g.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"g: dtype {g.dtype}, expected float32 or bfloat16")
    _need(g, None, name="g")
    M, N = g.shape[-2:]
    abc = [float(v) for step in steps for v in step]
    if len(abc) != 3 * len(steps):
        raise ValueError("steps: expected (a, b, c) for every step")
    return (math.prod(g.shape[:-2]), M, N, EP_DTYPE_F32 if g.dtype == torch.float32 else EP_DTYPE_BF16,
            (ctypes.c_float * max(1, len(abc)))(*abc))


def ep_orthogonalize(g, steps, out, workspace, eps=1e-7, status=None, stream=None):
    """out = Newton-Schulz orthogonalisation of every matrix of g [..., M, N] (bf16
    or fp32); steps: a sequence of (a, b, c), one a step.  out bf16, may be g;
    workspace: alloc_orthogonalize_workspace.  A wait that ran out is told by
    status alone."""
    count, M, N, dtype, abc = _stack(g, steps)
    _need(out, torch.bfloat16, g.shape, "out")
    _need(workspace, torch.uint8, name="workspace")
    if status is not None:
        _need(status, torch.int32, (1,), "status")
    _here(g, out, workspace, status)
    rc = load().ep_orthogonalize(_ptr(g), dtype, count, M, N, len(steps), abc, eps, _ptr(out),
                                 _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream))
    _check(rc, "ep_orthogonalize")


def ep_muon_update(g, m, w, w16, steps, workspace, lr, scale=1.0, momentum=0.95, nesterov=True,
                   weight_decay=0.0, eps=1e-7, status=None, stream=None):
    """One Muon step on a stack of weights [..., M, N], in place: momentum m and
    weights w (fp32), their bf16 copy w16 (may be None), from the gradient g (bf16
    or fp32).  steps and workspace as for ep_orthogonalize.  A wait that ran out is told
    by status alone; m, w and w16 then hold updated numbers and numbers as they were."""
    count, M, N, dtype, abc = _stack(g, steps)
    _need(m, torch.float32, g.shape, "m")
    _need(w, torch.float32, g.shape, "w")
    _need(w16, torch.bfloat16, g.shape, "w16", optional=True)
    _need(workspace, torch.uint8, name="workspace")
    if status is not None:
        _need(status, torch.int32, (1,), "status")
    _here(g, m, w, w16, workspace, status)
    rc = load().ep_muon_update(_ptr(g), dtype, _ptr(m), _ptr(w), _ptr(w16), count, M, N, lr, scale,
                               momentum, int(nesterov), weight_decay, len(steps), abc, eps,
                               _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream))
    _check(rc, "ep_muon_update")


def ep_read_status(status, stream=None) -> int:
    _need(status, torch.int32, (1,), "status")
    v = ctypes.c_int32(0)
    rc = load().ep_read_status(_ptr(status), ctypes.byref(v), _stream(stream))
    _check(rc, "ep_read_status")
    return int(v.value)


def ep_host_wait_counters(counters: torch.Tensor, timeout_ms: int) -> int:
    """Bounded host wait on host int64 counters (returns the EP code)."""
    if counters.is_cuda or counters.dtype != torch.int64 or not counters.is_contiguous():
        raise ValueError("counters must be a contiguous host int64 tensor")
    return int(load().ep_host_wait_counters(_ptr(counters), counters.numel(), timeout_ms))


def ep_format_e4m3(x, out, stream=None):
    """fp32 -> E4M3 bytes as the FP8 dispatch casts (x float32, out uint8)."""
    _need(x, torch.float32, name="x")
    _need(out, torch.uint8, tuple(x.shape), "out")
    _check(load().ep_format_e4m3(_ptr(x), _ptr(out), x.numel(), _stream(stream)), "ep_format_e4m3")


def ep_format_bf16(x, out, stream=None):
    """fp32 -> bf16 as the combine rounds (x float32, out bfloat16 or int16)."""
    _need(x, torch.float32, name="x")
    if out.dtype not in (torch.bfloat16, torch.int16):
        raise ValueError("out must be bfloat16 or int16")
    _need(out, None, tuple(x.shape), "out")
    _check(load().ep_format_bf16(_ptr(x), _ptr(out), x.numel(), _stream(stream)), "ep_format_bf16")


def ep_set_num_sms(num_sms: int) -> None:
    """SM budget of the data kernels (0: every SM)."""
    _check(load().ep_set_num_sms(int(num_sms)), "ep_set_num_sms")


def ep_get_num_sms() -> int:
    return int(load().ep_get_num_sms())


def ep_launch_count() -> int:
    return int(load().ep_launch_count())


# ------------------------------------------------------------------ allocation helpers

def alloc_layout(R: int, T_r: int, k: int, E: int, device="cuda"):
    i32 = dict(dtype=torch.int32, device=device)
    return dict(
        num_tokens_per_rank=torch.empty((R, R), **i32),
        num_tokens_per_expert=torch.empty((R, E), **i32),
        is_token_in_rank=torch.empty((R, T_r, R), dtype=torch.uint8, device=device),
        slot_rank=torch.empty((R, T_r, k), **i32),
    )


def alloc_notify(R: int, E: int, device="cuda"):
    i32 = dict(dtype=torch.int32, device=device)
    return dict(
        rank_prefix_matrix=torch.empty((R, R), **i32),
        expert_prefix=torch.empty((R + 1, E), **i32),
        num_recv_tokens_per_expert=torch.empty((R, E // R), **i32),
        psum=torch.empty((R, E // R + 1), dtype=torch.int64, device=device),
    )


def alloc_dispatch(R: int, T_r: int, H: int, k: int, fp8_mode: int, cap_rows: int, device="cuda"):
    rdt = torch.bfloat16 if fp8_mode == EP_FP8_NONE else torch.uint8
    return dict(
        recv_x=torch.empty((R, cap_rows, H), dtype=rdt, device=device),
        recv_scales=(None if fp8_mode == EP_FP8_NONE else
                     torch.empty((R, H // 128, cap_rows), dtype=_scale_dtype(fp8_mode),
                                 device=device)),
        recv_src_idx=torch.empty((R, cap_rows), dtype=torch.int32, device=device),
        combine_idx=torch.empty((R, T_r, k), dtype=torch.int32, device=device),
    )


def alloc_ll(R: int, T_r: int, H: int, E: int, k: int, max_tokens_per_rank: int, fp8_mode: int,
             device="cuda"):
    E_l = E // R
    S = R * max_tokens_per_rank
    rdt = torch.bfloat16 if fp8_mode == EP_FP8_NONE else torch.uint8
    return dict(
        packed_recv_x=torch.empty((R, E_l, S, H), dtype=rdt, device=device),
        packed_recv_scales=(None if fp8_mode == EP_FP8_NONE else
                            torch.empty((R, E_l, H // 128, S), dtype=_scale_dtype(fp8_mode),
                                        device=device)),
        packed_recv_src_info=torch.empty((R, E_l, S), dtype=torch.int32, device=device),
        layout_range=torch.empty((R, E_l, R), dtype=torch.int64, device=device),
        recv_count=torch.zeros((R, E_l), dtype=torch.int32, device=device),
        combine_idx=torch.empty((R, T_r, k), dtype=torch.int32, device=device),
    )


def alloc_workspace(R: int, T_r: int, k: int, E: int, H: int, device="cuda", stream=None):
    """Workspace for layout and dispatch (ep_workspace_size), cleaned and ready."""
    ws = torch.empty((ep_workspace_size(R, T_r, k, E, H),), dtype=torch.uint8, device=device)
    ep_clean_ll_buffer(None, R, E, ws, stream=stream)
    return ws


def alloc_moe_few_workspace(R: int, T_r: int, k: int, E: int, I: int, device="cuda"):
    """Workspace of ep_moe_few."""
    return torch.empty((ep_moe_few_workspace_size(R, T_r, k, E, I),), dtype=torch.uint8,
                       device=device)


def alloc_orthogonalize_workspace(shape, device="cuda"):
    """Workspace of ep_orthogonalize and ep_muon_update for a stack [..., M, N]."""
    size = ep_orthogonalize_workspace_size(math.prod(shape[:-2]), shape[-2], shape[-1])
    return torch.empty((size,), dtype=torch.uint8, device=device)


class LowLatencyBuffers:
    """The low-latency mode's two receive buffers (DeepEP's LL buffer holds
    the results of at most two low-latency calls at once): two sets of
    alloc_ll outputs, each with its own workspace, handed out in turn, so
    the received data of call i stays valid while call i+1 dispatches into
    the other set; call i+2 reuses the first.  Allocation only: the calls
    themselves are the ep_ll_* entry points, issued in stream order (the
    single-launch dispatch needs every SM, so two of them must not run
    concurrently on different streams)."""

    def __init__(self, R: int, T_r: int, H: int, E: int, k: int, max_tokens_per_rank: int,
                 fp8_mode: int, device="cuda", stream=None):
        self.sets = []
        for _ in range(2):
            b = alloc_ll(R, T_r, H, E, k, max_tokens_per_rank, fp8_mode, device=device)
            b["workspace"] = alloc_workspace(R, T_r, k, E, H, device=device, stream=stream)
            self.sets.append(b)
        self._turn = 0

    def next(self) -> dict:
        """The set for the next call (alternates 0, 1, 0, ...)."""
        b = self.sets[self._turn]
        self._turn ^= 1
        return b
