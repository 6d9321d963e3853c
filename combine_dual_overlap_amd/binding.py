"""ctypes binding of libdbomoe.so: the C ABI of include/dbomoe.h, same names.

Argument marshalling only: tensors become device pointers, streams become
hipStream_t handles, and a non-zero moe_status becomes a MoEError.  Every step
of the layer runs in the library's HIP kernels; there is no fallback path.  If
the library is not built, loading raises instead of degrading.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdbomoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_MISALIGNED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = \
    0, -1, -2, -3, -4, -5
MOE_F32, MOE_BF16, MOE_FP8_E4M3FN, MOE_INT8 = 0, 1, 2, 3
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
DBO_SCHED_UNSPLIT, DBO_SCHED_SERIAL, DBO_SCHED_DBO, DBO_SCHED_DBO_LATE_EVENT, DBO_SCHED_DBO_RECV_HOOK = 0, 1, 2, 3, 4
MOE_GEMM_NT, MOE_GEMM_NN, MOE_GEMM_TN = 0, 1, 2
MOE_GATE_NONE, MOE_GATE_CHANNEL, MOE_GATE_TOKEN, MOE_GATE_FULL = 0, 1, 2, 3
GEMM_KINDS = {"nt": MOE_GEMM_NT, "nn": MOE_GEMM_NN, "tn": MOE_GEMM_TN}
SCHEDULES = {"unsplit": 0, "serial": 1, "dbo": 2, "dbo_late_event": 3, "dbo_recv_hook": 4}

EXPORTED = [
    "moe_route_workspace_size", "moe_route_topk", "moe_dispatch_workspace_size", "moe_dispatch",
    "moe_get_device_error", "moe_ffn_workspace_size", "moe_ffn_auto_tile", "moe_grouped_ffn", "moe_combine",
    "dbo_ctx_create", "dbo_ctx_destroy", "dbo_ctx_set_timing", "dbo_ctx_ffn_times", "dbo_ctx_comm_times",
    "dbo_ctx_last_stats",
    "moe_layer_workspace_size", "moe_layer_workspace_layout", "dbo_moe_layer", "moe_status_string",
    "moe_quant_fp8_rows", "moe_dispatch_fp8", "moe_ffn_fp8_workspace_size", "moe_grouped_ffn_fp8",
    "moe_dispatch_send", "moe_dispatch_recv", "moe_dispatch_noalloc_max_workspace", "moe_dispatch_noalloc",
    "moe_grouped_gemm_workspace_size", "moe_grouped_gemm", "moe_grouped_swiglu", "moe_grouped_swiglu_backward",
    "moe_combine_backward", "moe_route_backward", "moe_adamw_table_size", "moe_adamw_table_build",
    "moe_adamw_table_check", "moe_adamw_step",
    "moe_route_select", "moe_route_balanced", "moe_route_bias_update", "moe_route_balance_loss_workspace_size",
    "moe_route_balance_loss", "moe_quant_int8_rows", "moe_dispatch_int8", "moe_grouped_gemm_int8",
    "moe_grouped_swiglu_int8", "moe_ffn_int8_workspace_size", "moe_grouped_ffn_int8", "moe_pre_norm", "moe_post_norm",
    "moe_combine_post_norm", "moe_norm_backward_workspace_size", "moe_pre_norm_backward", "moe_post_norm_backward",
]


class moe_route_params(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("k", ctypes.c_int32), ("score", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("n_groups", ctypes.c_int32),
                ("topk_groups", ctypes.c_int32), ("group_topn", ctypes.c_int32),
                ("routed_scale", ctypes.c_float)]


class moe_post_norm_params(ctypes.Structure):
    _fields_ = [("post_w", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("gate_kind", ctypes.c_int32),
                ("scale", ctypes.c_float), ("eps", ctypes.c_float), ("next_w", ctypes.c_void_p)]


class moe_block_params(ctypes.Structure):
    _fields_ = [("pre_w", ctypes.c_void_p), ("post", moe_post_norm_params), ("residual", ctypes.c_int32)]


class moe_layer_desc(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("I", ctypes.c_int32), ("act", ctypes.c_int32),
                ("wdt", ctypes.c_int32), ("route", moe_route_params),
                ("expert_begin", ctypes.c_int32), ("expert_end", ctypes.c_int32),
                ("w_router", ctypes.c_void_p), ("w13", ctypes.c_void_p), ("w2", ctypes.c_void_p),
                ("w13_scale", ctypes.c_void_p), ("w2_scale", ctypes.c_void_p),
                ("shared_I", ctypes.c_int32), ("shared_w13", ctypes.c_void_p),
                ("shared_w2", ctypes.c_void_p), ("fp8_act", ctypes.c_int32),
                ("select_bias", ctypes.c_void_p), ("block", ctypes.POINTER(moe_block_params))]


class dbo_opts(ctypes.Structure):
    _fields_ = [("schedule", ctypes.c_int32), ("min_tokens_to_split", ctypes.c_int32),
                ("split_at", ctypes.c_int32), ("comm_cu_budget", ctypes.c_int32),
                ("ffn_tile_m", ctypes.c_int32)]


class moe_adamw_tensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("master", ctypes.c_void_p), ("n", ctypes.c_int64), ("param_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("state_dtype", ctypes.c_int32)]


class moe_adamw_params(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("seed", ctypes.c_uint32)]


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


_LIB = None
_vp, _i32, _i64, _sz, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


def lib():
    """The loaded library.  Raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m combine_dual_overlap_amd.build` (no fallback path exists)")
        L = ctypes.CDLL(LIB_PATH)
        sig = {
            "moe_route_workspace_size": (_sz, [_i64, _i32, _i32]),
            "moe_route_topk": (_i32, [_vp, _i32, _i64, _i32, _vp, _vp, _vp, ctypes.POINTER(moe_route_params),
                                      _vp, _vp, _vp, _vp, _sz, _vp]),
            "moe_dispatch_workspace_size": (_sz, [_i64, _i32, _i32]),
            "moe_dispatch": (_i32, [_vp, _i32, _i64, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                                    _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
            "moe_get_device_error": (_i32, [_vp, ctypes.POINTER(_i32), _vp]),
            "moe_dispatch_noalloc_max_workspace": (_sz, []),
            "moe_dispatch_noalloc": (_i32, [_vp, _i32, _i64, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                                            _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
            "moe_ffn_workspace_size": (_sz, [_i64, _i32, _i32]),
            "moe_ffn_auto_tile": (_i32, [_i32, _i32, _i32, _i32, _i64, _i64, _i32]),
            "moe_grouped_ffn": (_i32, [_vp, _i32, _i32, _i32, _vp, _i32, _i64, _vp, _vp, _i32, _vp, _vp,
                                       _vp, _i32, _vp, _sz, _vp]),
            "moe_combine": (_i32, [_vp, _i32, _i64, _i32, _i32, _vp, _vp, _vp, _vp, _vp]),
            "dbo_ctx_create": (_i32, [ctypes.POINTER(_vp)]),
            "dbo_ctx_destroy": (None, [_vp]),
            "dbo_ctx_set_timing": (_i32, [_vp, _i32]),
            "dbo_ctx_ffn_times": (_i32, [_vp, _i32, ctypes.POINTER(ctypes.c_float)]),
            "dbo_ctx_comm_times": (_i32, [_vp, _i32, ctypes.POINTER(ctypes.c_float)]),
            "dbo_ctx_last_stats": (_i32, [_vp, ctypes.POINTER(_i64)]),
            "moe_layer_workspace_size": (_sz, [ctypes.POINTER(moe_layer_desc), _i64]),
            "moe_layer_workspace_layout": (_i32, [ctypes.POINTER(moe_layer_desc), _i64, _i32,
                                                  ctypes.POINTER(_i64)]),
            "dbo_moe_layer": (_i32, [_vp, ctypes.POINTER(moe_layer_desc), _vp, _i64, _vp, _vp, _vp,
                                     ctypes.POINTER(dbo_opts), _vp, _sz, _vp, _vp]),
            "moe_status_string": (ctypes.c_char_p, [_i32]),
            "moe_quant_fp8_rows": (_i32, [_vp, _i64, _i32, _vp, _vp, _vp]),
            "moe_dispatch_fp8": (_i32, [_vp, _i64, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                                        _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
            "moe_ffn_fp8_workspace_size": (_sz, [_i64, _i32]),
            "moe_dispatch_send": (_i32, [_vp, _i64, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp,
                                         _vp, _sz, _vp]),
            "moe_dispatch_recv": (_i32, [_vp, _i32, _i64, _i32, _i32, _vp, _vp, _vp, _vp]),
            "moe_grouped_ffn_fp8": (_i32, [_vp, _vp, _i32, _i32, _vp, _i32, _i64, _vp, _vp, _vp, _vp,
                                           _vp, _i32, _vp, _sz, _vp]),
            "moe_grouped_gemm_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i64, _i32, _i32]),
            "moe_grouped_gemm": (_i32, [_i32, _vp, _vp, _i32, _vp, _i32, _i64, _i32, _i32, _vp, _i32, _i32, _vp,
                                        _sz, _vp]),
            "moe_grouped_swiglu": (_i32, [_vp, _vp, _i32, _vp, _i32, _i64, _i32, _i32, _vp, _vp, _vp]),
            "moe_grouped_swiglu_backward": (_i32, [_vp, _vp, _vp, _i32, _vp, _i32, _i64, _i32, _i32, _vp, _vp]),
            "moe_combine_backward": (_i32, [_vp, _vp, _i32, _i64, _i32, _i32, _i64, _vp, _vp, _vp, _vp, _vp]),
            "moe_route_backward": (_i32, [_vp, _i64, _vp, _vp, ctypes.POINTER(moe_route_params), _vp, _i32, _vp]),
            "moe_adamw_table_size": (_sz, [_i32]),
            "moe_adamw_table_build": (_i32, [ctypes.POINTER(moe_adamw_tensor), _i32, _vp, _sz]),
            "moe_adamw_table_check": (_i32, [_vp]),
            "moe_adamw_step": (_i32, [_vp, _vp, ctypes.POINTER(moe_adamw_params), _vp, _vp, _vp, _vp]),
            "moe_route_select": (_i32, [_vp, _i64, _vp, ctypes.POINTER(moe_route_params), _vp, _vp, _vp, _vp]),
            "moe_route_balanced": (_i32, [_vp, _i32, _i64, _i32, _vp, _vp, _vp, ctypes.POINTER(moe_route_params),
                                          _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
            "moe_route_bias_update": (_i32, [_vp, _vp, _i32, _f32, _vp]),
            "moe_route_balance_loss_workspace_size": (_sz, [_i64, _i32]),
            "moe_route_balance_loss": (_i32, [_vp, _i64, _vp, ctypes.POINTER(moe_route_params), _f32, _vp, _vp, _i32,
                                              _i32, _vp, _sz, _vp]),
            "moe_quant_int8_rows": (_i32, [_vp, _i32, _i64, _i32, _vp, _vp, _vp]),
            "moe_dispatch_int8": (_i32, [_vp, _i32, _i64, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                                         _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
            "moe_grouped_gemm_int8": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _vp, _i32, _vp]),
            "moe_grouped_swiglu_int8": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _vp, _i32, _vp]),
            "moe_ffn_int8_workspace_size": (_sz, [_i64, _i32]),
            "moe_grouped_ffn_int8": (_i32, [_vp, _vp, _i32, _i32, _vp, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                            _vp]),
            "moe_pre_norm": (_i32, [_vp, _i32, _i64, _i32, _vp, _f32, _vp, _vp, _vp]),
            "moe_post_norm": (_i32, [_vp, _i32, _i64, _i32, _vp, ctypes.POINTER(moe_post_norm_params), _vp, _vp, _vp,
                                     _vp, _vp]),
            "moe_combine_post_norm": (_i32, [_vp, _i32, _i64, _i32, _i32, _vp, _vp, _vp, _vp,
                                             ctypes.POINTER(moe_post_norm_params), _vp, _vp, _vp, _vp, _vp, _vp]),
            "moe_norm_backward_workspace_size": (_sz, [_i64, _i32]),
            "moe_pre_norm_backward": (_i32, [_vp, _vp, _i32, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _sz,
                                             _vp]),
            "moe_post_norm_backward": (_i32, [_vp, _vp, _i32, _i64, _i32, _vp, ctypes.POINTER(moe_post_norm_params),
                                              _vp, _vp, _vp, _i32, _vp, _sz, _vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _LIB = L
    return _LIB


def status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoEError(status, where)


def ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a device tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return MOE_FP8_E4M3FN
    if t.dtype == torch.int8:
        return MOE_INT8
    raise ValueError(f"unsupported dtype {t.dtype}")


def stream_handle(s=None):
    if s is None:
        s = torch.cuda.current_stream()
    return s.cuda_stream


def route_params(E, k, score="softmax", renormalize=False, n_groups=1, topk_groups=1, group_topn=2,
                 routed_scale=1.0) -> moe_route_params:
    return moe_route_params(E, k, MOE_SCORE_SOFTMAX if score == "softmax" else MOE_SCORE_SIGMOID,
                            int(bool(renormalize)), n_groups, topk_groups if n_groups > 1 else 1,
                            group_topn if n_groups > 1 else 1, float(routed_scale))


# ------------------------------------------------------------------ entry points

def moe_route_workspace_size(T: int, H: int, E: int) -> int:
    return lib().moe_route_workspace_size(T, H, E)


def moe_route_topk(x, w_router, params: moe_route_params, topk_ids, topk_w, ws, logits_out=None,
                   logit_bias=None, forced_ids=None, stream=None):
    T, H = x.shape
    _check(lib().moe_route_topk(ptr(x), dtype_code(x), T, H, ptr(w_router), ptr(logit_bias), ptr(forced_ids),
                                ctypes.byref(params), ptr(logits_out), ptr(topk_ids), ptr(topk_w), ptr(ws),
                                ws.numel() * ws.element_size(), stream_handle(stream)), "moe_route_topk")


def moe_dispatch_workspace_size(T: int, k: int, E_loc: int) -> int:
    return lib().moe_dispatch_workspace_size(T, k, E_loc)


def moe_dispatch(x, topk_ids, E_total, expert_begin, expert_end, counts, offsets, perm, inv, x_perm, ws,
                 tile_m=0, tile_offsets=None, stream=None):
    T, H = x.shape
    k = topk_ids.shape[1] if topk_ids.dim() == 2 else 1
    _check(lib().moe_dispatch(ptr(x), dtype_code(x), T, H, ptr(topk_ids), k, E_total, expert_begin, expert_end,
                              tile_m, ptr(counts), ptr(offsets), ptr(tile_offsets), ptr(perm), ptr(inv),
                              ptr(x_perm), ptr(ws), ws.numel() * ws.element_size(), stream_handle(stream)),
           "moe_dispatch")


def moe_dispatch_noalloc_max_workspace() -> int:
    return lib().moe_dispatch_noalloc_max_workspace()


def moe_dispatch_noalloc(x, topk_ids, E_total, expert_begin, expert_end, counts, offsets, perm, inv, x_perm,
                         tile_m=0, tile_offsets=None, stream=None):
    T, H = x.shape
    k = topk_ids.shape[1] if topk_ids.dim() == 2 else 1
    _check(lib().moe_dispatch_noalloc(ptr(x), dtype_code(x), T, H, ptr(topk_ids), k, E_total, expert_begin,
                                      expert_end, tile_m, ptr(counts), ptr(offsets), ptr(tile_offsets), ptr(perm),
                                      ptr(inv), ptr(x_perm), stream_handle(stream)), "moe_dispatch_noalloc")


def moe_dispatch_send(topk_ids, E_total, expert_begin, expert_end, counts, offsets, perm, inv, ws, tile_m=0,
                      tile_offsets=None, stream=None):
    T = topk_ids.shape[0]
    k = topk_ids.shape[1] if topk_ids.dim() == 2 else 1
    _check(lib().moe_dispatch_send(ptr(topk_ids), T, k, E_total, expert_begin, expert_end, tile_m, ptr(counts),
                                   ptr(offsets), ptr(tile_offsets), ptr(perm), ptr(inv), ptr(ws),
                                   ws.numel() * ws.element_size(), stream_handle(stream)), "moe_dispatch_send")


def moe_dispatch_recv(x, k, inv, x_perm, xq_scale=None, stream=None):
    T, H = x.shape
    _check(lib().moe_dispatch_recv(ptr(x), dtype_code(x), T, H, k, ptr(inv), ptr(x_perm), ptr(xq_scale),
                                   stream_handle(stream)), "moe_dispatch_recv")


def moe_get_device_error(dispatch_ws, stream=None) -> int:
    code = ctypes.c_int32(0)
    _check(lib().moe_get_device_error(ptr(dispatch_ws), ctypes.byref(code), stream_handle(stream)),
           "moe_get_device_error")
    return code.value


def moe_ffn_workspace_size(cap_rows: int, I: int, act: int) -> int:
    return lib().moe_ffn_workspace_size(cap_rows, I, act)


def moe_ffn_auto_tile(act: int, wdt: int, H: int, I: int, rows_per_expert: int, rows1: int = 0,
                      I1: int = 0) -> int:
    return lib().moe_ffn_auto_tile(act, wdt, H, I, rows_per_expert, rows1, I1)


def moe_grouped_ffn(x_perm, I, offsets, E_loc, w13, w2, y_perm, ws, w13_scale=None, w2_scale=None,
                    tile_m=0, cap_rows=None, stream=None):
    cap = x_perm.shape[0] if cap_rows is None else cap_rows
    H = x_perm.shape[1]
    _check(lib().moe_grouped_ffn(ptr(x_perm), dtype_code(x_perm), H, I, ptr(offsets), E_loc, cap, ptr(w13),
                                 ptr(w2), dtype_code(w13), ptr(w13_scale), ptr(w2_scale), ptr(y_perm), tile_m,
                                 ptr(ws), ws.numel() * ws.element_size(), stream_handle(stream)),
           "moe_grouped_ffn")


def moe_quant_fp8_rows(x, q, scale, stream=None):
    n, K = x.shape
    _check(lib().moe_quant_fp8_rows(ptr(x), n, K, ptr(q), ptr(scale), stream_handle(stream)), "moe_quant_fp8_rows")


def moe_dispatch_fp8(x, topk_ids, E_total, expert_begin, expert_end, counts, offsets, perm, inv, xq_perm,
                     xq_scale, ws, tile_m=0, tile_offsets=None, stream=None):
    T, H = x.shape
    k = topk_ids.shape[1] if topk_ids.dim() == 2 else 1
    _check(lib().moe_dispatch_fp8(ptr(x), T, H, ptr(topk_ids), k, E_total, expert_begin, expert_end, tile_m,
                                  ptr(counts), ptr(offsets), ptr(tile_offsets), ptr(perm), ptr(inv), ptr(xq_perm),
                                  ptr(xq_scale), ptr(ws), ws.numel() * ws.element_size(), stream_handle(stream)),
           "moe_dispatch_fp8")


def moe_ffn_fp8_workspace_size(cap_rows: int, I: int) -> int:
    return lib().moe_ffn_fp8_workspace_size(cap_rows, I)


def moe_grouped_ffn_fp8(xq_perm, xq_scale, I, offsets, E_loc, w13, w2, w13_scale, w2_scale, y_perm, ws,
                        tile_m=0, cap_rows=None, stream=None):
    cap = xq_perm.shape[0] if cap_rows is None else cap_rows
    H = xq_perm.shape[1]
    _check(lib().moe_grouped_ffn_fp8(ptr(xq_perm), ptr(xq_scale), H, I, ptr(offsets), E_loc, cap, ptr(w13),
                                     ptr(w2), ptr(w13_scale), ptr(w2_scale), ptr(y_perm), tile_m, ptr(ws),
                                     ws.numel() * ws.element_size(), stream_handle(stream)),
           "moe_grouped_ffn_fp8")


def moe_combine(y_perm, T, k, inv, topk_w, out, shared_out=None, stream=None):
    H = out.shape[1]
    _check(lib().moe_combine(ptr(y_perm), dtype_code(out), T, H, k, ptr(inv), ptr(topk_w), ptr(shared_out),
                             ptr(out), stream_handle(stream)), "moe_combine")


# ------------------------------------------------------------------ training
# The calls below check shapes, types and devices, and run on the tensors'
# device: `stream` defaults to that device's current stream.  A decode-sized
# call takes the GPU less time than these checks took with torch.device and
# torch.cuda.Stream objects, so devices are compared by number and the stream
# is taken as a raw handle.

def _need(ok, what: str):
    if not ok:
        raise ValueError(what)


def _device(t) -> int:
    d = t.get_device()
    if d < 0:
        raise ValueError("expected a device tensor")
    return d


def _ptrs(d: int, *ts) -> list:
    """Addresses of contiguous tensors on device d; None stays None."""
    out = []
    for t in ts:
        if t is None:
            out.append(None)
            continue
        if t.get_device() != d:
            raise ValueError("tensors on different devices" if t.is_cuda else "expected a device tensor")
        if not t.is_contiguous():
            raise ValueError("expected a contiguous tensor")
        out.append(t.data_ptr())
    return out


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(fn: str, d: int, stream, *args):
    f = getattr(_LIB or lib(), fn)
    if d == _current_device():          # (a tensor on d: CUDA is initialised)
        h = stream.cuda_stream if stream is not None else _raw_stream(d) if _raw_stream else stream_handle()
        st = f(*args, h)
    else:
        with torch.cuda.device(d):
            st = f(*args, stream_handle(stream))
    if st != MOE_OK:
        raise MoEError(st, fn)


_CODES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.uint8: MOE_FP8_E4M3FN,
          torch.float8_e4m3fn: MOE_FP8_E4M3FN}


def _code(dtype) -> int:
    c = _CODES.get(dtype)
    if c is None:
        raise ValueError(f"unsupported dtype {dtype}")
    return c


def _groups(offsets, experts: int) -> int:
    """E_loc of a grouped call: offsets [E_loc + 1] int32, or None for one dense group."""
    if offsets is None:
        if experts != 1:
            raise ValueError("offsets None: one group")
        return 1
    if offsets.dtype != torch.int32 or offsets.shape != (experts + 1,):
        raise ValueError(f"offsets: expected int32 [{experts + 1}]")
    return experts


def _gemm_sizes(kind: str, a, b, offsets, c):
    """(kind code, E_loc, cap_rows, N, K) of a moe_grouped_gemm call, shapes and types checked."""
    code, sa, sb, sc = GEMM_KINDS.get(kind), a.shape, b.shape, c.shape
    if code is None:
        raise ValueError(f"kind: one of {sorted(GEMM_KINDS)}")
    if a.dtype != b.dtype or len(sa) != 2:
        raise ValueError("a: a 2-d tensor of b's type")
    if code == MOE_GEMM_TN:
        if len(sc) != 3 or sa != (sa[0], sc[1]) or sb != (sa[0], sc[2]):
            raise ValueError("tn: a [rows, N], b [rows, K], c [E, N, K]")
        E, N, K = sc
    else:
        if len(sb) != 3 or len(sc) != 2 or sc[0] != sa[0]:
            raise ValueError(f"{kind}: a [rows, K], b of 3 axes, c [rows, N]")
        E, N, K = sb[0], sc[1], sa[1]
        if (sb[1], sb[2]) != ((N, K) if code == MOE_GEMM_NT else (K, N)):
            raise ValueError(f"{kind}: b [E, N, K] (nt) or [E, K, N] (nn)")
    return code, _groups(offsets, E), sa[0], N, K


def moe_grouped_gemm_workspace_size(kind: str, a, b, offsets, c) -> int:
    """Bytes of workspace of moe_grouped_gemm on these tensors (0: none needed)."""
    code, E, cap, N, K = _gemm_sizes(kind, a, b, offsets, c)
    return lib().moe_grouped_gemm_workspace_size(code, _code(a.dtype), int(offsets is None), E, cap, N, K)


# No call's workspace is larger: a split product has fewer than 512 tiles of at most 128 x 128 fp32 partial sums.
GEMM_MAX_WORKSPACE = 512 * 128 * 128 * 4


def moe_grouped_gemm(kind: str, a, b, offsets, c, ws=None, accumulate=False, stream=None):
    """Matrix products grouped by expert; rows [offsets[e], offsets[e+1]) belong to expert e.

    "nt": c [rows, N] = a [rows, K] b[e]^T, b [E, N, K].  "nn": the same with b [E, K, N].
    "tn": c [E, N, K] = a[rows of e]^T b[rows of e], a [rows, N], b [rows, K].
    offsets None: one group of all rows.  accumulate: c += product."""
    code, E, cap, N, K = _gemm_sizes(kind, a, b, offsets, c)
    d = _device(a)
    pa, pb, po, pc, pw = _ptrs(d, a, b, offsets, c, ws)
    _call("moe_grouped_gemm", d, stream, code, pa, pb, _code(a.dtype), po, E, cap, N, K, pc, _code(c.dtype),
          1 if accumulate else 0, pw, 0 if ws is None else ws.nbytes)


def moe_grouped_swiglu(x_perm, w13, offsets, h, gu=None, stream=None):
    """h [rows, I] = silu(x g^T) * (x u^T) with w13 [E, 2I, H]; gu [rows, 2I] (optional) gets the pre-activations."""
    rows, H = x_perm.shape
    E, I = w13.shape[0], h.shape[1]
    if w13.shape != (E, 2 * I, H) or h.shape != (rows, I) or (gu is not None and gu.shape != (rows, 2 * I)):
        raise ValueError("w13 [E, 2I, H], h [rows, I], gu [rows, 2I]")
    t = x_perm.dtype
    if w13.dtype != t or h.dtype != t or (gu is not None and gu.dtype != t):
        raise ValueError("one type for every tensor")
    d = _device(x_perm)
    px, pw, po, pg, ph = _ptrs(d, x_perm, w13, offsets, gu, h)
    _call("moe_grouped_swiglu", d, stream, px, pw, _code(t), po, _groups(offsets, E), rows, H, I, pg, ph)


def moe_grouped_swiglu_backward(dy_perm, w2, gu, offsets, dgu, stream=None):
    """dgu [rows, 2I] from dy_perm [rows, H], w2 [E, H, I] and the pre-activations gu [rows, 2I] (dgu may be gu)."""
    rows, H = dy_perm.shape
    E, I = w2.shape[0], w2.shape[2]
    if w2.shape != (E, H, I) or gu.shape != (rows, 2 * I) or dgu.shape != (rows, 2 * I):
        raise ValueError("dy_perm [rows, H], w2 [E, H, I], gu and dgu [rows, 2I]")
    t = dy_perm.dtype
    if w2.dtype != t or gu.dtype != t or dgu.dtype != t:
        raise ValueError("one type for every tensor")
    d = _device(dy_perm)
    py, pw, pg, po, pd = _ptrs(d, dy_perm, w2, gu, offsets, dgu)
    _call("moe_grouped_swiglu_backward", d, stream, py, pw, pg, _code(t), po, _groups(offsets, E), rows, H, I, pd)


def moe_combine_backward(dout, y_perm, inv, topk_w, dy_perm, dtopk_w, stream=None):
    """dy_perm [rows, H] and dtopk_w [T, k] of moe_combine's out [T, H]; inv [T*k], topk_w [T, k] as it took them."""
    T, H = dout.shape
    k, cap = topk_w.shape[1], y_perm.shape[0]
    if y_perm.shape != (cap, H) or dy_perm.shape != (cap, H):
        raise ValueError("y_perm and dy_perm [rows, H]")
    t = dout.dtype
    if y_perm.dtype != t or dy_perm.dtype != t:
        raise ValueError("one type for dout, y_perm and dy_perm")
    if topk_w.shape != (T, k) or dtopk_w.shape != (T, k) or inv.numel() != T * k:
        raise ValueError("topk_w, dtopk_w, inv: T x k")
    if inv.dtype != torch.int32 or topk_w.dtype != torch.float32 or dtopk_w.dtype != torch.float32:
        raise ValueError("inv int32; weights float32")
    d = _device(dout)
    po, py, pi, pw, pd, pg = _ptrs(d, dout, y_perm, inv, topk_w, dy_perm, dtopk_w)
    _call("moe_combine_backward", d, stream, po, py, _code(t), T, H, k, cap, pi, pw, pd, pg)


def moe_route_backward(logits, topk_ids, dtopk_w, params: moe_route_params, dlogits, stream=None):
    """dlogits [T, E] (float32 or bfloat16) of moe_route_topk's weights, from its logits, ids and dtopk_w [T, k]."""
    T, E = logits.shape
    k = params.k
    if E != params.E or dlogits.shape != (T, E):
        raise ValueError("logits and dlogits [T, E] with params.E experts")
    if topk_ids.shape != (T, k) or dtopk_w.shape != (T, k):
        raise ValueError("topk_ids and dtopk_w [T, k]")
    if logits.dtype != torch.float32 or dtopk_w.dtype != torch.float32 or topk_ids.dtype != torch.int32:
        raise ValueError("logits and dtopk_w float32, topk_ids int32")
    d = _device(logits)
    pl, pi, pw, pd = _ptrs(d, logits, topk_ids, dtopk_w, dlogits)
    _call("moe_route_backward", d, stream, pl, T, pi, pw, params, pd, _code(dlogits.dtype))


def adamw_params(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, seed=0) -> moe_adamw_params:
    return moe_adamw_params(lr, beta1, beta2, eps, weight_decay, seed & 0xFFFFFFFF)


class AdamWTable:
    """The tensors of an optimizer as moe_adamw_step takes them: the table on the host and its copy on the device.
    Holds references: the tensors live as long as it."""

    def __init__(self, host, device_copy, device: int, keep):
        self.host, self.device_copy, self.device, self.keep = host, device_copy, device, keep
        self.host_ptr, self.device_ptr = host.data_ptr(), device_copy.data_ptr()


def moe_adamw_table(params, grads, m, v, m_scale=None, v_scale=None, master=None) -> AdamWTable:
    """Lists of tensors, one entry per parameter.  params float32 or bfloat16; grads likewise; m and v float32, or
    8-bit codes (float8_e4m3fn or uint8) with m_scale and v_scale uint8 [ceil(n / 128)]; master float32 or None.
    Made once (it copies the table to the device); the tensors must stay where they are."""
    n = len(params)
    _need(n > 0, "no tensors")
    cols = [None if c is None else list(c) for c in (params, grads, m, v, m_scale, v_scale, master)]
    for c in cols:
        _need(c is None or len(c) == n, "lists of one length")
    none = [None] * n
    entries = (moe_adamw_tensor * n)()
    f32, bf16, floats = torch.float32, torch.bfloat16, (torch.float32, torch.bfloat16)
    d = None
    for i, (p, g, mi, vi, ms, vs, ma) in enumerate(zip(*(none if c is None else c for c in cols))):
        size, t, gt, mt = p.numel(), p.dtype, g.dtype, mi.dtype
        d = _device(p) if d is None else d
        if g.numel() != size or mi.numel() != size or vi.numel() != size or (ma is not None and ma.numel() != size):
            raise ValueError(f"tensor {i}: sizes differ")
        if (t not in floats or gt not in floats or mt != vi.dtype or (mt != f32 and _CODES.get(mt) != MOE_FP8_E4M3FN)
                or (ma is not None and (ma.dtype != f32 or t != bf16))):
            raise ValueError(f"tensor {i}: types")
        if (mt != f32) != (ms is not None) or (ms is None) != (vs is None):
            raise ValueError(f"tensor {i}: scales go with 8-bit states")
        if ms is not None and (ms.dtype != torch.uint8 or vs.dtype != torch.uint8 or
                               not ms.numel() == vs.numel() == (size + 127) // 128):
            raise ValueError(f"tensor {i}: scales uint8 [ceil(n / 128)]")
        entries[i] = moe_adamw_tensor(*_ptrs(d, p, g, mi, vi, ms, vs, ma), size, _CODES[t], _CODES[gt], _CODES[mt])
    nbytes = lib().moe_adamw_table_size(n)
    host = torch.zeros(nbytes, dtype=torch.uint8)
    _check(lib().moe_adamw_table_build(entries, n, host.data_ptr(), nbytes), "moe_adamw_table_build")
    _check(lib().moe_adamw_table_check(host.data_ptr()), "moe_adamw_table_check")
    return AdamWTable(host, host.to(torch.device("cuda", d)), d, cols)


def moe_adamw_step(table: AdamWTable, hp: moe_adamw_params, step, lr_scale=None, grad_scale=None, stream=None):
    """One update of the table's tensors.  step: int32 device scalar, 1 at the first update; lr_scale and grad_scale:
    float32 device scalars or None."""
    if step.dtype != torch.int32 or step.numel() != 1:
        raise ValueError("step: one int32")
    for s in (lr_scale, grad_scale):
        if s is not None and (s.dtype != torch.float32 or s.numel() != 1):
            raise ValueError("lr_scale, grad_scale: one float32")
    d = table.device
    _call("moe_adamw_step", d, stream, table.host_ptr, table.device_ptr, hp, *_ptrs(d, step, lr_scale, grad_scale))


# ------------------------------------------------------------------ balanced routing
# (with the checks, devices and streams of the training calls)

def _nbytes(ws) -> int:
    return 0 if ws is None else ws.nbytes


def _typed(t, dtype, shape, what: str):
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{what}: {dtype} {list(shape)}")


def _check_select(E, T, params, topk_ids, topk_w, select_bias, load):
    k = params.k
    if E != params.E:
        raise ValueError("logits of params.E experts")
    if (topk_ids.dtype != torch.int32 or topk_ids.shape != (T, k) or topk_w.dtype != torch.float32 or
            topk_w.shape != (T, k)):
        raise ValueError(f"topk_ids int32, topk_w float32 [{T}, {k}]")
    if select_bias is not None and (select_bias.dtype != torch.float32 or select_bias.shape != (E,)):
        raise ValueError(f"select_bias: float32 [{E}]")
    if load is not None and (load.dtype != torch.int32 or load.shape != (E,)):
        raise ValueError(f"load: int32 [{E}]")


def moe_route_select(logits, params: moe_route_params, topk_ids, topk_w, select_bias=None, load=None, stream=None):
    """topk_ids and topk_w [T, k] of logits [T, E] float32: chosen by score + select_bias [E], weighted by the score.
    load [E] int32 (optional): the number of tokens of each expert is added."""
    T, E = logits.shape
    if logits.dtype != torch.float32:
        raise ValueError("logits: float32")
    _check_select(E, T, params, topk_ids, topk_w, select_bias, load)
    d = _device(logits)
    pl, pb, pi, pw, po = _ptrs(d, logits, select_bias, topk_ids, topk_w, load)
    _call("moe_route_select", d, stream, pl, T, pb, params, pi, pw, po)


def moe_route_balanced(x, w_router, params: moe_route_params, topk_ids, topk_w, ws, select_bias=None, load=None,
                       logits_out=None, logit_bias=None, stream=None):
    """moe_route_topk with moe_route_select's selection: x [T, H], w_router [E, H]."""
    T, H = x.shape
    E = w_router.numel() // H
    if w_router.dtype != x.dtype or w_router.shape[-2:] != (E, H):
        raise ValueError("w_router: [E, H] of x's type")
    _check_select(E, T, params, topk_ids, topk_w, select_bias, load)
    if logits_out is not None:
        _typed(logits_out, torch.float32, (T, E), "logits_out")
    if logit_bias is not None:
        _typed(logit_bias, torch.float32, (E,), "logit_bias")
    d = _device(x)
    px, pr, pl, pb, pg, pi, pw, po, ps = _ptrs(d, x, w_router, logit_bias, select_bias, logits_out, topk_ids, topk_w,
                                               load, ws)
    _call("moe_route_balanced", d, stream, px, _code(x.dtype), T, H, pr, pl, pb, params, pg, pi, pw, po, ps, _nbytes(ws))


def moe_route_bias_update(bias, load, rate: float, stream=None):
    """bias [E] float32 += rate * sign(mean load - load); load [E] int32 becomes zero."""
    E = bias.numel()
    _typed(bias, torch.float32, (E,), "bias")
    _typed(load, torch.int32, (E,), "load")
    d = _device(bias)
    pb, pl = _ptrs(d, bias, load)
    _call("moe_route_bias_update", d, stream, pb, pl, E, rate)


def moe_route_balance_loss_workspace_size(T: int, E: int) -> int:
    return lib().moe_route_balance_loss_workspace_size(T, E)


def moe_route_balance_loss(logits, load, params: moe_route_params, coef: float, loss, dlogits, ws, accumulate=False,
                           stream=None):
    """loss [1] = coef * E * sum_e (load_e / sum load) mean_t q_te and its gradient dlogits [T, E] (accumulate: added)."""
    T, E = logits.shape
    _typed(logits, torch.float32, (T, E), "logits")
    _typed(load, torch.int32, (E,), "load")
    if E != params.E or loss.dtype != torch.float32 or loss.numel() != 1 or dlogits.shape != (T, E):
        raise ValueError("logits and dlogits [T, params.E], loss one float32")
    d = _device(logits)
    pl, pn, po, pd, pw = _ptrs(d, logits, load, loss, dlogits, ws)
    _call("moe_route_balance_loss", d, stream, pl, T, pn, params, coef, po, pd, _code(dlogits.dtype),
          1 if accumulate else 0, pw, _nbytes(ws))


# ------------------------------------------------------------------ 8-bit integers

def moe_quant_int8_rows(x, q, scale, stream=None):
    """x [..., K] float32 or bfloat16 -> q int8 of its shape and scale [...] float32: x = q * scale of its row."""
    K, n = x.shape[-1], scale.numel()
    _typed(q, torch.int8, x.shape, "q")
    _typed(scale, torch.float32, x.shape[:-1], "scale")
    d = _device(x)
    px, pq, ps = _ptrs(d, x, q, scale)
    _call("moe_quant_int8_rows", d, stream, px, _code(x.dtype), n, K, pq, ps)


def moe_dispatch_int8(x, topk_ids, E_total, expert_begin, expert_end, counts, offsets, perm, inv, xq_perm, xq_scale, ws,
                      tile_m=0, tile_offsets=None, stream=None):
    """moe_dispatch whose rows arrive as 8-bit integers xq_perm [T*k, H] with scales xq_scale [T*k]."""
    T, H = x.shape
    k = topk_ids.shape[1]
    E_loc = expert_end - expert_begin
    i32 = torch.int32
    _typed(topk_ids, i32, (T, k), "topk_ids")
    for t, n, what in ((counts, E_loc, "counts"), (offsets, E_loc + 1, "offsets"), (perm, T * k, "perm"), (inv, T * k, "inv")):
        if t.dtype != i32 or t.numel() < n:
            raise ValueError(f"{what}: int32 [{n}]")
    if tile_offsets is not None and (tile_offsets.dtype != i32 or tile_offsets.numel() < E_loc + 1):
        raise ValueError(f"tile_offsets: int32 [{E_loc + 1}]")
    if xq_perm.dtype != torch.int8 or xq_perm.numel() < T * k * H or xq_scale.dtype != torch.float32 or xq_scale.numel() < T * k:
        raise ValueError(f"xq_perm int8 [{T * k}, {H}], xq_scale float32 [{T * k}]")
    d = _device(x)
    px, pi, pc, po, pt, pp, pv, pq, ps, pw = _ptrs(d, x, topk_ids, counts, offsets, tile_offsets, perm, inv, xq_perm,
                                                   xq_scale, ws)
    _call("moe_dispatch_int8", d, stream, px, _code(x.dtype), T, H, pi, k, E_total, expert_begin, expert_end, tile_m,
          pc, po, pt, pp, pv, pq, ps, pw, _nbytes(ws))


def moe_grouped_gemm_int8(a, a_scale, b, b_scale, offsets, c, stream=None):
    """c [rows, N] = (a [rows, K] b[e]^T) * a_scale [rows] * b_scale[e], b int8 [E, N, K]; offsets None: one group."""
    (rows, K), (E, N, _) = a.shape, b.shape
    _typed(b, torch.int8, (E, N, K), "b")
    _typed(a, torch.int8, (rows, K), "a")
    _typed(a_scale, torch.float32, (rows,), "a_scale")
    _typed(b_scale, torch.float32, (E, N), "b_scale")
    if c.shape != (rows, N):
        raise ValueError(f"c: [{rows}, {N}]")
    d = _device(a)
    pa, ps, pb, pt, po, pc = _ptrs(d, a, a_scale, b, b_scale, offsets, c)
    _call("moe_grouped_gemm_int8", d, stream, pa, ps, pb, pt, po, _groups(offsets, E), rows, N, K, pc, _code(c.dtype))


def moe_grouped_swiglu_int8(xq, xq_scale, w13, w13_scale, offsets, h, stream=None):
    """h [rows, I] = silu(g) * u of the products of xq [rows, H] with w13 int8 [E, 2I, H] and their scales."""
    (rows, H), I, E = xq.shape, h.shape[1], w13.shape[0]
    _typed(xq, torch.int8, (rows, H), "xq")
    _typed(xq_scale, torch.float32, (rows,), "xq_scale")
    _typed(w13, torch.int8, (E, 2 * I, H), "w13")
    _typed(w13_scale, torch.float32, (E, 2 * I), "w13_scale")
    if h.shape != (rows, I):
        raise ValueError(f"h: [{rows}, {I}]")
    d = _device(xq)
    px, ps, pw, pt, po, ph = _ptrs(d, xq, xq_scale, w13, w13_scale, offsets, h)
    _call("moe_grouped_swiglu_int8", d, stream, px, ps, pw, pt, po, _groups(offsets, E), rows, H, I, ph, _code(h.dtype))


def moe_ffn_int8_workspace_size(cap_rows: int, I: int) -> int:
    return lib().moe_ffn_int8_workspace_size(cap_rows, I)


def moe_grouped_ffn_int8(xq, xq_scale, offsets, w13, w13_scale, w2, w2_scale, y, ws, stream=None):
    """y [rows, H] bfloat16: SwiGLU experts in 8-bit integers; w13 [E, 2I, H], w2 [E, H, I] int8 with a scale per row."""
    (rows, H), (E, _, I) = xq.shape, w2.shape
    _typed(xq, torch.int8, (rows, H), "xq")
    _typed(xq_scale, torch.float32, (rows,), "xq_scale")
    _typed(w13, torch.int8, (E, 2 * I, H), "w13")
    _typed(w13_scale, torch.float32, (E, 2 * I), "w13_scale")
    _typed(w2, torch.int8, (E, H, I), "w2")
    _typed(w2_scale, torch.float32, (E, H), "w2_scale")
    _typed(y, torch.bfloat16, (rows, H), "y")
    d = _device(xq)
    px, ps, po, pa, pb, p2, p3, py, pw = _ptrs(d, xq, xq_scale, offsets, w13, w13_scale, w2, w2_scale, y, ws)
    _call("moe_grouped_ffn_int8", d, stream, px, ps, H, I, po, _groups(offsets, E), rows, pa, p2, pb, p3, py, pw,
          _nbytes(ws))


# ------------------------------------------------------------------ norms before and after the layer

# (Each check is one expression: a decode-sized call takes the GPU 5 us, and a function
# call for every tensor took the host as long.)

def _gate_kind(gate, T: int, H: int, dtype) -> int:
    """By shape: [H] and [T, H] of the rows' type, or [T, 1] float32."""
    s, t = gate.shape, gate.dtype
    if t == dtype and s == (H,):
        return MOE_GATE_CHANNEL
    if t == torch.float32 and s == (T, 1) and H != 1:
        return MOE_GATE_TOKEN
    if t == dtype and s == (T, H):
        return MOE_GATE_FULL
    raise ValueError(f"gate: {dtype} [{H}] or [{T}, {H}], or float32 [{T}, 1]")


def moe_pre_norm(x, w, n, eps: float, rstd=None, stream=None):
    """n [T, H] = x / rms(x) * w; rstd [T] float32 (optional): 1 / rms, for the backward pass.  n may be x."""
    t, s = x.dtype, x.shape
    T, H = s
    if n.dtype != t or n.shape != s or w.dtype != t or w.shape != (H,):
        raise ValueError(f"n: {t} [{T}, {H}], w: {t} [{H}]")
    if rstd is not None and (rstd.dtype != torch.float32 or rstd.shape != (T,)):
        raise ValueError(f"rstd: float32 [{T}]")
    d = _device(x)
    px, pw, pn, pr = _ptrs(d, x, w, n, rstd)
    _call("moe_pre_norm", d, stream, px, _code(t), T, H, pw, eps, pn, pr)


def _check_post(t, s, post_w, next_w, next_n, rstd, next_rstd):
    T, H = s
    if ((post_w is not None and (post_w.dtype != t or post_w.shape != (H,))) or
            (next_w is not None and (next_w.dtype != t or next_w.shape != (H,)))):
        raise ValueError(f"post_w, next_w: {t} [{H}]")
    if next_n is not None and (next_n.dtype != t or next_n.shape != s):
        raise ValueError(f"next_n: {t} [{T}, {H}]")
    if ((rstd is not None and (rstd.dtype != torch.float32 or rstd.shape != (T,))) or
            (next_rstd is not None and (next_rstd.dtype != torch.float32 or next_rstd.shape != (T,)))):
        raise ValueError(f"rstd, next_rstd: float32 [{T}]")


def moe_post_norm(y, res, out, eps: float, post_w=None, gate=None, scale: float = 1.0, rstd=None, next_w=None,
                  next_n=None, next_rstd=None, stream=None):
    """out [T, H] = res + scale * gate * (y / rms(y) * post_w), and next_n = out / rms(out) * next_w.

    res None: no residual; post_w None: no norm; gate [H] or [T, H] of y's type, or float32 [T, 1].  out may be res."""
    t, s = y.dtype, y.shape
    T, H = s
    if out.dtype != t or out.shape != s or (res is not None and (res.dtype != t or res.shape != s)):
        raise ValueError(f"res, out: {t} [{T}, {H}]")
    _check_post(t, s, post_w, next_w, next_n, rstd, next_rstd)
    kind = MOE_GATE_NONE if gate is None else _gate_kind(gate, T, H, t)
    d = _device(y)
    py, pe, po, pr, pn, ps, pw, pg, px = _ptrs(d, y, res, out, rstd, next_n, next_rstd, post_w, gate, next_w)
    _call("moe_post_norm", d, stream, py, _code(t), T, H, pe, moe_post_norm_params(pw, pg, kind, scale, eps, px), po, pr,
          pn, ps)


def moe_combine_post_norm(y_perm, inv, topk_w, res, out, eps: float, post_w=None, gate=None, scale: float = 1.0,
                          shared_out=None, y_out=None, rstd=None, next_w=None, next_n=None, next_rstd=None, stream=None):
    """moe_post_norm of moe_combine's sum of y_perm, inv [T*k], topk_w [T, k] (+ shared_out [T, H]); y_out: that sum."""
    t, s = out.dtype, out.shape
    T, H = s
    k = topk_w.shape[1]
    if y_perm.dtype != t or y_perm.dim() != 2 or y_perm.shape[1] != H:
        raise ValueError(f"y_perm: {t} [rows, {H}]")
    if topk_w.dtype != torch.float32 or topk_w.shape != (T, k) or inv.dtype != torch.int32 or inv.numel() != T * k:
        raise ValueError("topk_w float32 [T, k], inv int32 [T * k]")
    if ((res is not None and (res.dtype != t or res.shape != s)) or
            (shared_out is not None and (shared_out.dtype != t or shared_out.shape != s)) or
            (y_out is not None and (y_out.dtype != t or y_out.shape != s))):
        raise ValueError(f"res, shared_out, y_out: {t} [{T}, {H}]")
    _check_post(t, s, post_w, next_w, next_n, rstd, next_rstd)
    kind = MOE_GATE_NONE if gate is None else _gate_kind(gate, T, H, t)
    d = _device(out)
    pp, pi, pk, ph, pe, po, py, pr, pn, ps, pw, pg, px = _ptrs(d, y_perm, inv, topk_w, shared_out, res, out, y_out, rstd,
                                                               next_n, next_rstd, post_w, gate, next_w)
    _call("moe_combine_post_norm", d, stream, pp, _code(t), T, H, k, pi, pk, ph, pe,
          moe_post_norm_params(pw, pg, kind, scale, eps, px), po, py, pr, pn, ps)


def moe_norm_backward_workspace_size(T: int, H: int) -> int:
    return lib().moe_norm_backward_workspace_size(T, H)


def moe_pre_norm_backward(dn, x, rstd, w, dx, dw, ws, dres=None, accumulate=False, stream=None):
    """dx [T, H] = dres + the gradient of moe_pre_norm's x; dw [H] float32 (or None).  dx may be dn or dres."""
    t, s = x.dtype, x.shape
    T, H = s
    if (dn.dtype != t or dn.shape != s or dx.dtype != t or dx.shape != s or
            (dres is not None and (dres.dtype != t or dres.shape != s))):
        raise ValueError(f"dn, dx, dres: {t} [{T}, {H}]")
    if w.dtype != t or w.shape != (H,) or rstd.dtype != torch.float32 or rstd.shape != (T,):
        raise ValueError(f"w: {t} [{H}], rstd: float32 [{T}]")
    if dw is not None and (dw.dtype != torch.float32 or dw.shape != (H,)):
        raise ValueError(f"dw: float32 [{H}]")
    d = _device(x)
    pd, px, pr, pw, pe, po, pg, ps = _ptrs(d, dn, x, rstd, w, dres, dx, dw, ws)
    _call("moe_pre_norm_backward", d, stream, pd, px, _code(t), T, H, pr, pw, pe, po, pg, 1 if accumulate else 0, ps,
          _nbytes(ws))


def moe_post_norm_backward(dout, y, dy, ws, rstd=None, post_w=None, dpost_w=None, gate=None, dgate=None,
                           scale: float = 1.0, accumulate=False, stream=None):
    """Gradients of moe_post_norm's out: dy [T, H], dpost_w [H] float32 (or None), dgate (or None): float32 [H] or
    [T, 1], or [T, H] of y's type, as the gate.  The residual's gradient is dout."""
    t, s = y.dtype, y.shape
    T, H = s
    if dout.dtype != t or dout.shape != s or dy.dtype != t or dy.shape != s:
        raise ValueError(f"dout, dy: {t} [{T}, {H}]")
    _check_post(t, s, post_w, None, None, rstd, None)
    kind = MOE_GATE_NONE if gate is None else _gate_kind(gate, T, H, t)
    if dpost_w is not None and (dpost_w.dtype != torch.float32 or dpost_w.shape != (H,)):
        raise ValueError(f"dpost_w: float32 [{H}]")
    if dgate is not None and (gate is None or dgate.dtype != (t if kind == MOE_GATE_FULL else torch.float32) or
                              dgate.shape != gate.shape):
        raise ValueError("dgate: of the gate's shape, float32 (a full gate's: of its type)")
    d = _device(y)
    pd, py, po, ps, pr, pw, pc, pg, pt = _ptrs(d, dout, y, dy, ws, rstd, post_w, dpost_w, gate, dgate)
    _call("moe_post_norm_backward", d, stream, pd, py, _code(t), T, H, pr,
          moe_post_norm_params(pw, pg, kind, scale, 1.0, None), po, pc, pt, 1 if accumulate else 0, ps, _nbytes(ws))


class DboContext:
    """Owns a dbo_ctx (the per-microbatch HIP events)."""

    def __init__(self):
        h = ctypes.c_void_p()
        _check(lib().dbo_ctx_create(ctypes.byref(h)), "dbo_ctx_create")
        self.handle = h

    def close(self):
        if self.handle:
            lib().dbo_ctx_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_timing(self, enable: bool):
        _check(lib().dbo_ctx_set_timing(self.handle, int(enable)), "dbo_ctx_set_timing")

    def ffn_times(self, back: int = 0):
        """[A gate/up, A down, B gate/up, B down] ms of the timed call `back` calls ago."""
        ms = (ctypes.c_float * 4)()
        _check(lib().dbo_ctx_ffn_times(self.handle, back, ms), "dbo_ctx_ffn_times")
        return list(ms)

    def comm_times(self, back: int = 0):
        """[A dispatch, B dispatch, A combine, B combine] ms of the timed call `back` calls ago."""
        ms = (ctypes.c_float * 4)()
        _check(lib().dbo_ctx_comm_times(self.handle, back, ms), "dbo_ctx_comm_times")
        return list(ms)

    def last_stats(self) -> dict:
        s = (ctypes.c_int64 * 6)()
        _check(lib().dbo_ctx_last_stats(self.handle, s), "dbo_ctx_last_stats")
        return dict(schedule=s[0], T0=s[1], yields_a=s[2], yields_b=s[3], stages=s[4], records=s[5])


def moe_layer_workspace_size(desc: moe_layer_desc, T_max: int) -> int:
    return lib().moe_layer_workspace_size(ctypes.byref(desc), T_max)


def moe_layer_workspace_layout(desc: moe_layer_desc, T: int, mb: int) -> dict:
    off = (ctypes.c_int64 * 12)()
    _check(lib().moe_layer_workspace_layout(ctypes.byref(desc), T, mb, off), "moe_layer_workspace_layout")
    names = ["logits", "topk_ids", "topk_w", "counts", "offsets", "tile_offsets", "perm", "inv", "x_perm",
             "y_perm", "shared_out", "dispatch_ws"]
    return dict(zip(names, list(off)))


def dbo_moe_layer(ctx: DboContext, desc: moe_layer_desc, x, out, opts: dbo_opts, ws, compute_stream=None,
                  comm_stream=None, forced_ids=None, logit_bias=None):
    T = x.shape[0]
    _check(lib().dbo_moe_layer(ctx.handle, ctypes.byref(desc), ptr(x), T, ptr(forced_ids), ptr(logit_bias),
                               ptr(out), ctypes.byref(opts), ptr(ws), ws.numel() * ws.element_size(),
                               stream_handle(compute_stream), stream_handle(comm_stream)), "dbo_moe_layer")
