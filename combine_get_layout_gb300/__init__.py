"""Python binding of libep_gb300.so (MoE dispatch / combine layout on GB300,
with the router gate before it and experts' products inside).

Two layers, both argument marshalling only -- every step of layout, dispatch
and combine runs in the library's CUDA kernels:

* ``ep_*`` functions with the C ABI's names and arguments (include/ep.h),
  taking ``EpConfig`` / ``EpLayout`` ctypes structures and raw pointers.
* A torch layer (``Config``, ``Layout``, ``get_layout``, ``dispatch``,
  ``combine``, ``route``, ``expert_w4``, ``expert_mm``, ...) that allocates device
  buffers with torch, passes ``tensor.data_ptr()`` and the current CUDA stream, and raises ``EpError``
  on a non-zero status.  torch provides memory and streams, nothing else.
  The calls of the router gate, of the experts' products and of the
  activation between them go through a small compiled extension (ep_torch_calls) instead of ctypes.

There is no fallback: if the shared library is missing, importing this
package raises.  Build it with ``python combine_get_layout_gb300/build_lib.py``.
"""

from __future__ import annotations

import ctypes
import dataclasses
import os
from threading import Lock as _Lock, get_ident as _get_ident
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libep_gb300.so")

EP_OK = 0
EP_ERR_INVALID_ARG = 1
EP_ERR_EXPERT_RANGE = 2
EP_ERR_DUP_EXPERT = 3
EP_ERR_CAPACITY = 4
EP_ERR_CUDA = 5
EP_ERR_TIMEOUT = 6
EP_ERR_TIMEOUT_PENDING = 7

EP_GRAD_BF16 = 0
EP_GRAD_FP32 = 1
EP_GRAD_FP32_ADD = 2

# The entry points include/ep.h declares (kept in sync by a test).
ABI_SYMBOLS = (
    "ep_recv_capacity",
    "ep_layout_workspace_bytes",
    "ep_get_layout",
    "ep_dispatch",
    "ep_combine",
    "ep_layout_and_dispatch",
    "ep_scale_ld",
    "ep_dispatch_fp8",
    "ep_combine_epilogue",
    "ep_dispatch_backward",
    "ep_combine_backward",
    "ep_rank_rows_capacity",
    "ep_dispatch_ranks",
    "ep_expand",
    "ep_reduce_ranks",
    "ep_combine_ranks",
    "ep_dispatch_from_host",
    "ep_combine_to_host",
    "ep_route",
    "ep_route_workspace_bytes",
    "ep_route_balance",
    "ep_route_backward",
    "ep_w4_codes_bytes",
    "ep_w4_scales_bytes",
    "ep_w4_zeros_bytes",
    "ep_w4_pack",
    "ep_expert_w4",
    "ep_expert_mm",
    "ep_expert_mm_backward",
    "ep_selftest_expert_timeout",
    "ep_act_save",
    "ep_act_backward",
    "ep_check_error",
    "ep_selftest_wait_timeout",
    "ep_selftest_layout_timeout",
    "ep_selftest_fp8_quotient",
    "ep_last_cuda_error",
    "ep_get_layout_noalloc",
    "ep_status_str",
)


class EpConfig(ctypes.Structure):
    _fields_ = [
        ("max_tokens", ctypes.c_int32),
        ("hidden", ctypes.c_int32),
        ("num_topk", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("num_ranks", ctypes.c_int32),
        ("expert_alignment", ctypes.c_int32),
        ("use_fp8_dispatch", ctypes.c_int32),
        ("zero_padding", ctypes.c_int32),
    ]


class EpLayout(ctypes.Structure):
    _fields_ = [
        ("expert_count", ctypes.c_void_p),
        ("expert_start", ctypes.c_void_p),
        ("expert_end", ctypes.c_void_p),
        ("rank_start", ctypes.c_void_p),
        ("tokens_per_rank", ctypes.c_void_p),
        ("is_token_in_rank", ctypes.c_void_p),
        ("slot_of", ctypes.c_void_p),
        ("src_info", ctypes.c_void_p),
        ("err", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("rank_row_start", ctypes.c_void_p),
        ("rank_slot_of", ctypes.c_void_p),
        ("rank_src", ctypes.c_void_p),
        ("num_tokens", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class EpRouterConfig(ctypes.Structure):
    _fields_ = [
        ("num_experts", ctypes.c_int32),
        ("num_topk", ctypes.c_int32),
        ("score", ctypes.c_int32),
        ("num_groups", ctypes.c_int32),
        ("topk_groups", ctypes.c_int32),
        ("renormalize", ctypes.c_int32),
        ("logits_bf16", ctypes.c_int32),
        ("route_scale", ctypes.c_float),
    ]


class EpW4Config(ctypes.Structure):
    _fields_ = [
        ("num_experts", ctypes.c_int32),
        ("in_features", ctypes.c_int32),
        ("out_features", ctypes.c_int32),
        ("group_size", ctypes.c_int32),
        ("x_fp8", ctypes.c_int32),
        ("gated", ctypes.c_int32),
        ("has_zeros", ctypes.c_int32),
    ]


class EpExpertConfig(ctypes.Structure):
    _fields_ = [
        ("num_experts", ctypes.c_int32),
        ("in_features", ctypes.c_int32),
        ("out_features", ctypes.c_int32),
        ("x_fp8", ctypes.c_int32),
        ("gated", ctypes.c_int32),
    ]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with "
            "`python combine_get_layout_gb300/build_lib.py` (nvcc, sm_103a)")
    L = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    L.ep_recv_capacity.restype = i64
    L.ep_recv_capacity.argtypes = [P(EpConfig)]
    L.ep_layout_workspace_bytes.restype = i64
    L.ep_layout_workspace_bytes.argtypes = [P(EpConfig)]
    L.ep_get_layout.restype = i32
    L.ep_get_layout.argtypes = [P(EpConfig), i32, vp, P(EpLayout), vp, vp]
    L.ep_dispatch.restype = i32
    L.ep_dispatch.argtypes = [P(EpConfig), P(EpLayout), vp, vp, vp, vp, vp, vp]
    L.ep_combine.restype = i32
    L.ep_combine.argtypes = [P(EpConfig), P(EpLayout), vp, vp, vp, vp]
    L.ep_scale_ld.restype = i64
    L.ep_scale_ld.argtypes = [P(EpConfig)]
    L.ep_dispatch_fp8.restype = i32
    L.ep_dispatch_fp8.argtypes = [P(EpConfig), P(EpLayout), vp, vp, vp, vp, vp, vp, i32, vp, vp]
    L.ep_combine_epilogue.restype = i32
    L.ep_combine_epilogue.argtypes = [P(EpConfig), P(EpLayout), vp, vp, vp, vp, vp, vp, vp, vp]
    L.ep_dispatch_backward.restype = i32
    L.ep_dispatch_backward.argtypes = [P(EpConfig), P(EpLayout), vp, vp, vp, vp, vp]
    L.ep_combine_backward.restype = i32
    L.ep_combine_backward.argtypes = [P(EpConfig), P(EpLayout), vp, vp, vp, vp, vp, vp]
    L.ep_rank_rows_capacity.restype = i64
    L.ep_rank_rows_capacity.argtypes = [P(EpConfig)]
    L.ep_dispatch_ranks.restype = i32
    L.ep_dispatch_ranks.argtypes = [P(EpConfig), P(EpLayout), vp, vp, vp, vp, vp, vp, vp]
    L.ep_expand.restype = i32
    L.ep_expand.argtypes = [P(EpConfig), P(EpLayout), vp, vp, vp, vp, vp, vp]
    L.ep_reduce_ranks.restype = i32
    L.ep_reduce_ranks.argtypes = [P(EpConfig), P(EpLayout), vp, vp, vp, vp, vp]
    L.ep_combine_ranks.restype = i32
    L.ep_combine_ranks.argtypes = [P(EpConfig), P(EpLayout), vp, vp, vp]
    L.ep_layout_and_dispatch.restype = i32
    L.ep_layout_and_dispatch.argtypes = [P(EpConfig), i32, vp, P(EpLayout), vp, vp, vp, vp,
                                         vp, vp]
    L.ep_dispatch_from_host.restype = i32
    L.ep_dispatch_from_host.argtypes = [P(EpConfig), P(EpLayout), vp, vp, vp, vp, vp, vp,
                                        i32, vp]
    L.ep_combine_to_host.restype = i32
    L.ep_combine_to_host.argtypes = [P(EpConfig), P(EpLayout), vp, vp, vp, vp, i32, vp]
    L.ep_route.restype = i32
    L.ep_route.argtypes = [P(EpRouterConfig), i32, vp, i64, vp, vp, vp, vp, vp]
    L.ep_route_workspace_bytes.restype = i64
    L.ep_route_workspace_bytes.argtypes = [P(EpRouterConfig), i32]
    L.ep_route_balance.restype = i32
    L.ep_route_balance.argtypes = [P(EpRouterConfig), i32, vp, i64, vp, vp, i32, vp, vp, vp,
                                   vp, vp, vp, vp, vp, vp]
    L.ep_route_backward.restype = i32
    L.ep_route_backward.argtypes = [P(EpRouterConfig), i32, vp, i64, vp, vp, vp, i32, vp, vp,
                                    vp, vp, vp, i64, vp]
    for f in (L.ep_w4_codes_bytes, L.ep_w4_scales_bytes, L.ep_w4_zeros_bytes):
        f.restype = i64
        f.argtypes = [P(EpW4Config)]
    L.ep_w4_pack.restype = i32
    L.ep_w4_pack.argtypes = [P(EpW4Config), vp, vp, vp, vp, vp, vp, vp]
    L.ep_expert_w4.restype = i32
    L.ep_expert_w4.argtypes = [P(EpW4Config), i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.ep_expert_mm.restype = i32
    L.ep_expert_mm.argtypes = [P(EpExpertConfig), i32, i32, vp, vp, vp, vp, vp, vp, vp, vp]
    L.ep_selftest_expert_timeout.restype = i32
    L.ep_selftest_expert_timeout.argtypes = L.ep_expert_mm.argtypes
    L.ep_expert_mm_backward.restype = i32
    L.ep_expert_mm_backward.argtypes = [P(EpExpertConfig), i32, i32, vp, vp, vp, vp, vp, vp, vp,
                                        vp, i32, vp, vp]
    L.ep_act_save.restype = i32
    L.ep_act_save.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp]
    L.ep_act_backward.restype = i32
    L.ep_act_backward.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp]
    L.ep_check_error.restype = i32
    L.ep_check_error.argtypes = [P(EpLayout), vp]
    L.ep_selftest_fp8_quotient.restype = i32
    L.ep_selftest_fp8_quotient.argtypes = [vp, vp, vp]
    L.ep_selftest_wait_timeout.restype = i32
    L.ep_selftest_wait_timeout.argtypes = [i64, vp, vp]
    L.ep_selftest_layout_timeout.restype = i32
    L.ep_selftest_layout_timeout.argtypes = [P(EpConfig), i32, vp, P(EpLayout), i32, i64, vp]
    L.ep_get_layout_noalloc.restype = i32
    L.ep_get_layout_noalloc.argtypes = [P(EpConfig), i32, vp, P(EpLayout), vp, vp]
    L.ep_last_cuda_error.restype = i32
    L.ep_last_cuda_error.argtypes = []
    L.ep_status_str.restype = ctypes.c_char_p
    L.ep_status_str.argtypes = [i32]
    return L


_lib = _load()


def lib():
    """The loaded ctypes library (for tests that call the ABI directly)."""
    return _lib


# ---- C-ABI names ------------------------------------------------------------

def ep_recv_capacity(cfg: EpConfig) -> int:
    return int(_lib.ep_recv_capacity(ctypes.byref(cfg)))


def ep_layout_workspace_bytes(cfg: EpConfig) -> int:
    return int(_lib.ep_layout_workspace_bytes(ctypes.byref(cfg)))


def ep_get_layout(cfg, num_tokens, d_topk_idx, layout, h_expert_count, stream) -> int:
    return int(_lib.ep_get_layout(ctypes.byref(cfg), num_tokens, d_topk_idx,
                                  ctypes.byref(layout), h_expert_count, stream))


def ep_dispatch(cfg, layout, d_x, d_topk_weights, d_recv_x, d_recv_scale,
                d_recv_w, stream) -> int:
    return int(_lib.ep_dispatch(ctypes.byref(cfg), ctypes.byref(layout), d_x,
                                d_topk_weights, d_recv_x, d_recv_scale,
                                d_recv_w, stream))


def ep_combine(cfg, layout, d_expert_out, d_topk_weights, d_y, stream) -> int:
    return int(_lib.ep_combine(ctypes.byref(cfg), ctypes.byref(layout),
                               d_expert_out, d_topk_weights, d_y, stream))


def ep_scale_ld(cfg: EpConfig) -> int:
    return int(_lib.ep_scale_ld(ctypes.byref(cfg)))


def ep_dispatch_fp8(cfg, layout, d_x, d_x_q, d_x_scale, d_topk_weights, d_recv_q,
                    d_recv_scale, scale_col_major, d_recv_w, stream) -> int:
    return int(_lib.ep_dispatch_fp8(ctypes.byref(cfg), ctypes.byref(layout), d_x, d_x_q,
                                    d_x_scale, d_topk_weights, d_recv_q, d_recv_scale,
                                    int(scale_col_major), d_recv_w, stream))


def ep_combine_epilogue(cfg, layout, d_expert_out, d_topk_weights, d_bias0, d_bias1,
                        d_recv_w, d_y, d_combined_w, stream) -> int:
    return int(_lib.ep_combine_epilogue(ctypes.byref(cfg), ctypes.byref(layout),
                                        d_expert_out, d_topk_weights, d_bias0, d_bias1,
                                        d_recv_w, d_y, d_combined_w, stream))


def ep_dispatch_backward(cfg, layout, d_grad_recv, d_grad_recv_w, d_grad_x, d_grad_w,
                         stream) -> int:
    return int(_lib.ep_dispatch_backward(ctypes.byref(cfg), ctypes.byref(layout),
                                         d_grad_recv, d_grad_recv_w, d_grad_x, d_grad_w,
                                         stream))


def ep_combine_backward(cfg, layout, d_dy, d_topk_weights, d_expert_out,
                        d_grad_expert_out, d_grad_w, stream) -> int:
    return int(_lib.ep_combine_backward(ctypes.byref(cfg), ctypes.byref(layout), d_dy,
                                        d_topk_weights, d_expert_out, d_grad_expert_out,
                                        d_grad_w, stream))


def ep_rank_rows_capacity(cfg: EpConfig) -> int:
    return int(_lib.ep_rank_rows_capacity(ctypes.byref(cfg)))


def ep_dispatch_ranks(cfg, layout, d_x, d_topk_idx, d_topk_weights, d_rank_x,
                      d_rank_topk_idx, d_rank_topk_w, stream) -> int:
    return int(_lib.ep_dispatch_ranks(ctypes.byref(cfg), ctypes.byref(layout), d_x,
                                      d_topk_idx, d_topk_weights, d_rank_x,
                                      d_rank_topk_idx, d_rank_topk_w, stream))


def ep_expand(cfg, layout, d_topk_idx, d_rank_x, d_rank_topk_w, d_recv_x, d_recv_w,
              stream) -> int:
    return int(_lib.ep_expand(ctypes.byref(cfg), ctypes.byref(layout), d_topk_idx,
                              d_rank_x, d_rank_topk_w, d_recv_x, d_recv_w, stream))


def ep_reduce_ranks(cfg, layout, d_topk_idx, d_expert_out, d_topk_weights, d_rank_y,
                    stream) -> int:
    return int(_lib.ep_reduce_ranks(ctypes.byref(cfg), ctypes.byref(layout), d_topk_idx,
                                    d_expert_out, d_topk_weights, d_rank_y, stream))


def ep_combine_ranks(cfg, layout, d_rank_y, d_y, stream) -> int:
    return int(_lib.ep_combine_ranks(ctypes.byref(cfg), ctypes.byref(layout), d_rank_y,
                                     d_y, stream))


def ep_layout_and_dispatch(cfg, num_tokens, d_topk_idx, layout, d_x, d_topk_weights,
                           d_recv_x, d_recv_scale, d_recv_w, stream) -> int:
    return int(_lib.ep_layout_and_dispatch(ctypes.byref(cfg), int(num_tokens), d_topk_idx,
                                           ctypes.byref(layout), d_x, d_topk_weights, d_recv_x,
                                           d_recv_scale, d_recv_w, stream))


def ep_dispatch_from_host(cfg, layout, h_x, d_x, d_topk_weights, d_recv_x, d_recv_scale,
                          d_recv_w, num_chunks, stream) -> int:
    return int(_lib.ep_dispatch_from_host(ctypes.byref(cfg), ctypes.byref(layout), h_x, d_x,
                                          d_topk_weights, d_recv_x, d_recv_scale, d_recv_w,
                                          int(num_chunks), stream))


def ep_combine_to_host(cfg, layout, d_expert_out, d_topk_weights, d_y, h_y, num_chunks,
                       stream) -> int:
    return int(_lib.ep_combine_to_host(ctypes.byref(cfg), ctypes.byref(layout), d_expert_out,
                                       d_topk_weights, d_y, h_y, int(num_chunks), stream))


def ep_route(cfg, num_tokens, d_logits, ld_logits, d_bias, d_token_mask, d_topk_idx,
             d_topk_weights, stream) -> int:
    return _lib.ep_route(cfg, num_tokens, d_logits, ld_logits, d_bias, d_token_mask,
                         d_topk_idx, d_topk_weights, stream)


def ep_route_workspace_bytes(cfg: EpRouterConfig, num_seqs: int) -> int:
    return _lib.ep_route_workspace_bytes(cfg, num_seqs)


def ep_route_balance(cfg, num_tokens, d_logits, ld_logits, d_bias, d_token_mask, num_seqs,
                     d_seq_start, d_topk_idx, d_topk_weights, d_expert_count, d_expert_prob,
                     d_seq_tokens, d_loss, d_workspace, stream) -> int:
    return _lib.ep_route_balance(cfg, num_tokens, d_logits, ld_logits, d_bias, d_token_mask,
                                 num_seqs, d_seq_start, d_topk_idx, d_topk_weights,
                                 d_expert_count, d_expert_prob, d_seq_tokens, d_loss,
                                 d_workspace, stream)


def ep_route_backward(cfg, num_tokens, d_logits, ld_logits, d_token_mask, d_topk_idx, d_grad_w,
                      num_seqs, d_seq_start, d_expert_count, d_seq_tokens, d_grad_loss,
                      d_grad_logits, ld_grad, stream) -> int:
    return _lib.ep_route_backward(cfg, num_tokens, d_logits, ld_logits, d_token_mask,
                                  d_topk_idx, d_grad_w, num_seqs, d_seq_start, d_expert_count,
                                  d_seq_tokens, d_grad_loss, d_grad_logits, ld_grad, stream)


def ep_w4_codes_bytes(cfg: EpW4Config) -> int:
    return _lib.ep_w4_codes_bytes(cfg)


def ep_w4_scales_bytes(cfg: EpW4Config) -> int:
    return _lib.ep_w4_scales_bytes(cfg)


def ep_w4_zeros_bytes(cfg: EpW4Config) -> int:
    return _lib.ep_w4_zeros_bytes(cfg)


def ep_w4_pack(cfg, d_codes, d_scales, d_zeros, d_packed_codes, d_packed_scales,
               d_packed_zeros, stream) -> int:
    return _lib.ep_w4_pack(cfg, d_codes, d_scales, d_zeros, d_packed_codes, d_packed_scales,
                           d_packed_zeros, stream)


def ep_expert_w4(cfg, cap, num_rows, d_x, d_x_scale, d_codes, d_scales, d_zeros,
                 d_expert_start, d_expert_end, d_out, stream) -> int:
    return _lib.ep_expert_w4(cfg, cap, num_rows, d_x, d_x_scale, d_codes, d_scales, d_zeros,
                             d_expert_start, d_expert_end, d_out, stream)


def ep_expert_mm(cfg, cap, num_rows, d_x, d_x_scale, d_w, d_expert_start, d_expert_end, d_out,
                 d_err, stream) -> int:
    return _lib.ep_expert_mm(cfg, cap, num_rows, d_x, d_x_scale, d_w, d_expert_start,
                             d_expert_end, d_out, d_err, stream)


def ep_selftest_expert_timeout(cfg, cap, num_rows, d_x, d_x_scale, d_w, d_expert_start,
                               d_expert_end, d_out, d_err, stream) -> int:
    return _lib.ep_selftest_expert_timeout(cfg, cap, num_rows, d_x, d_x_scale, d_w,
                                           d_expert_start, d_expert_end, d_out, d_err, stream)


def ep_expert_mm_backward(cfg, cap, num_rows, d_grad_out, d_w, d_x, d_x_scale, d_expert_start,
                          d_expert_end, d_grad_x, d_grad_w, grad_w_type, d_err, stream) -> int:
    return _lib.ep_expert_mm_backward(cfg, cap, num_rows, d_grad_out, d_w, d_x, d_x_scale,
                                      d_expert_start, d_expert_end, d_grad_x, d_grad_w,
                                      grad_w_type, d_err, stream)


def ep_act_save(num_experts, width, cap, num_rows, d_h, d_expert_start, d_expert_end, d_a, d_q,
                d_scale, stream) -> int:
    return _lib.ep_act_save(num_experts, width, cap, num_rows, d_h, d_expert_start, d_expert_end,
                            d_a, d_q, d_scale, stream)


def ep_act_backward(num_experts, width, cap, num_rows, d_grad_a, d_q, d_scale, d_expert_start,
                    d_expert_end, d_grad_h, d_a, stream) -> int:
    return _lib.ep_act_backward(num_experts, width, cap, num_rows, d_grad_a, d_q, d_scale,
                                d_expert_start, d_expert_end, d_grad_h, d_a, stream)


def ep_check_error(layout, stream) -> int:
    return int(_lib.ep_check_error(ctypes.byref(layout), stream))


def ep_selftest_fp8_quotient(d_counts, d_first, stream) -> int:
    return int(_lib.ep_selftest_fp8_quotient(d_counts, d_first, stream))


def ep_selftest_wait_timeout(timeout_ns, d_err, stream) -> int:
    return int(_lib.ep_selftest_wait_timeout(int(timeout_ns), d_err, stream))


def ep_selftest_layout_timeout(cfg, num_tokens, d_topk_idx, layout, stall_tile, timeout_ns,
                               stream) -> int:
    return int(_lib.ep_selftest_layout_timeout(ctypes.byref(cfg), num_tokens, d_topk_idx,
                                               ctypes.byref(layout), int(stall_tile),
                                               int(timeout_ns), stream))


def ep_get_layout_noalloc(cfg, num_tokens, d_topk_idx, layout, h_expert_count,
                          stream) -> int:
    """ep_get_layout with the scratch in the library's own device memory
    (layout.workspace is ignored)."""
    return int(_lib.ep_get_layout_noalloc(ctypes.byref(cfg), num_tokens, d_topk_idx,
                                          ctypes.byref(layout), h_expert_count,
                                          stream))


def ep_last_cuda_error() -> int:
    return int(_lib.ep_last_cuda_error())


def ep_status_str(status: int) -> str:
    return _lib.ep_status_str(int(status)).decode()


# ---- torch layer ------------------------------------------------------------

class EpError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = int(status)
        msg = f"{what}: {ep_status_str(status)} ({status})"
        if self.status == EP_ERR_CUDA:
            self.cuda_error = ep_last_cuda_error()
            msg += f", cudaError {self.cuda_error}"
        super().__init__(msg)


def _check(status: int, what: str):
    if status != EP_OK:
        raise EpError(status, what)


@dataclasses.dataclass(frozen=True)
class Config:
    """Mirror of ep_config (see include/ep.h)."""

    max_tokens: int
    hidden: int
    num_topk: int
    num_experts: int
    num_ranks: int
    expert_alignment: int = 128
    use_fp8_dispatch: bool = False
    zero_padding: bool = False

    def c(self) -> EpConfig:
        return EpConfig(self.max_tokens, self.hidden, self.num_topk,
                        self.num_experts, self.num_ranks, self.expert_alignment,
                        int(self.use_fp8_dispatch), int(self.zero_padding))

    @property
    def capacity(self) -> int:
        cap = ep_recv_capacity(self.c())
        if cap < 0:
            raise EpError(EP_ERR_INVALID_ARG, "config")
        return cap


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


class Layout:
    """Device buffers of one layout handle, allocated with torch."""

    def __init__(self, cfg: Config, device="cuda", with_ranks: bool = False):
        import torch

        self.cfg = cfg
        E, R, K, T = cfg.num_experts, cfg.num_ranks, cfg.num_topk, cfg.max_tokens
        cap = cfg.capacity
        ws = ep_layout_workspace_bytes(cfg.c())
        i32 = dict(dtype=torch.int32, device=device)
        self.expert_count = torch.zeros(E, **i32)
        self.expert_start = torch.zeros(E + 1, **i32)
        self.expert_end = torch.zeros(E, **i32)
        self.rank_start = torch.zeros(R + 1, **i32)
        self.tokens_per_rank = torch.zeros(R, **i32)
        self.is_token_in_rank = torch.zeros((max(T, 1), R), dtype=torch.uint8, device=device)
        self.slot_of = torch.full((max(T, 1), K), -1, **i32)
        self.src_info = torch.full((cap, 2), -1, **i32)
        self.err = torch.zeros(4, **i32)
        self.workspace = torch.zeros(max(ws, 16), dtype=torch.uint8, device=device)
        self.rank_row_start = self.rank_slot_of = self.rank_src = None
        if with_ranks:
            self.rank_row_start = torch.zeros(R + 1, **i32)
            self.rank_slot_of = torch.full((max(T, 1), R), -1, **i32)
            self.rank_src = torch.full((max(T * min(K, R), 1),), -1, **i32)
        self.c = EpLayout(
            _ptr(self.expert_count), _ptr(self.expert_start), _ptr(self.expert_end),
            _ptr(self.rank_start), _ptr(self.tokens_per_rank),
            _ptr(self.is_token_in_rank), _ptr(self.slot_of), _ptr(self.src_info),
            _ptr(self.err), _ptr(self.workspace), _ptr(self.rank_row_start),
            _ptr(self.rank_slot_of), _ptr(self.rank_src), 0, 0)

    @property
    def num_tokens(self) -> int:
        return int(self.c.num_tokens)


def get_layout(cfg: Config, topk_idx, layout: Optional[Layout] = None,
               sync: bool = False, stream=None, with_ranks: bool = False) -> Layout:
    """ep_get_layout on an int64 CUDA tensor [T, K]."""
    import numpy as np

    if layout is None:
        layout = Layout(cfg, device=topk_idx.device, with_ranks=with_ranks)
    T = int(topk_idx.shape[0])
    h = None
    if sync:
        h = np.zeros(cfg.num_experts, np.int32)
    st = ep_get_layout(cfg.c(), T, _ptr(topk_idx.contiguous()) if T else None,
                       layout.c, None if h is None else h.ctypes.data_as(ctypes.c_void_p),
                       _stream(stream))
    _check(st, "ep_get_layout")
    layout.h_expert_count = h
    return layout


def dispatch(cfg: Config, layout: Layout, x, topk_weights=None, recv_x=None,
             recv_scale=None, recv_w=None, want_weights: bool = True, stream=None):
    """ep_dispatch.  x: bf16 CUDA tensor [T, H].  Returns (recv_x, recv_scale,
    recv_w); recv_x is bf16 [cap, H] or uint8 (E4M3 bits) [cap, H]."""
    import torch

    cap, H = cfg.capacity, cfg.hidden
    dev = x.device
    if recv_x is None:
        dt = torch.uint8 if cfg.use_fp8_dispatch else torch.bfloat16
        recv_x = torch.empty((cap, H), dtype=dt, device=dev)
    if cfg.use_fp8_dispatch and recv_scale is None:
        recv_scale = torch.empty((cap, H // 128), dtype=torch.float32, device=dev)
    if want_weights and topk_weights is not None and recv_w is None:
        recv_w = torch.empty(cap, dtype=torch.float32, device=dev)
    st = ep_dispatch(cfg.c(), layout.c, _ptr(x), _ptr(topk_weights), _ptr(recv_x),
                     _ptr(recv_scale), _ptr(recv_w), _stream(stream))
    _check(st, "ep_dispatch")
    return recv_x, recv_scale, recv_w


def combine(cfg: Config, layout: Layout, expert_out, topk_weights=None, y=None,
            stream=None):
    """ep_combine.  expert_out: bf16 CUDA tensor [cap, H]; returns bf16 [T, H]."""
    import torch

    T = layout.num_tokens
    if y is None:
        y = torch.empty((T, cfg.hidden), dtype=torch.bfloat16, device=expert_out.device)
    st = ep_combine(cfg.c(), layout.c, _ptr(expert_out), _ptr(topk_weights),
                    _ptr(y), _stream(stream))
    _check(st, "ep_combine")
    return y


def layout_and_dispatch(cfg: Config, topk_idx, x, topk_weights=None, layout=None,
                        recv_x=None, recv_scale=None, recv_w=None, want_weights: bool = True,
                        stream=None):
    """ep_layout_and_dispatch.  topk_idx: int64 CUDA tensor [T, K]; x: bf16 CUDA
    tensor [T, H].  Returns (layout, recv_x, recv_scale, recv_w)."""
    import torch

    cap, H = cfg.capacity, cfg.hidden
    dev = x.device
    L = layout or Layout(cfg, device=dev)
    if recv_x is None:
        dt = torch.uint8 if cfg.use_fp8_dispatch else torch.bfloat16
        recv_x = torch.empty((cap, H), dtype=dt, device=dev)
    if cfg.use_fp8_dispatch and recv_scale is None:
        recv_scale = torch.empty((cap, H // 128), dtype=torch.float32, device=dev)
    if want_weights and topk_weights is not None and recv_w is None:
        recv_w = torch.empty(cap, dtype=torch.float32, device=dev)
    st = ep_layout_and_dispatch(cfg.c(), topk_idx.shape[0], _ptr(topk_idx), L.c, _ptr(x),
                                _ptr(topk_weights), _ptr(recv_x), _ptr(recv_scale),
                                _ptr(recv_w), _stream(stream))
    _check(st, "ep_layout_and_dispatch")
    return L, recv_x, recv_scale, recv_w


def dispatch_from_host(cfg: Config, layout: Layout, h_x, d_x=None, topk_weights=None,
                       recv_x=None, recv_scale=None, recv_w=None, want_weights: bool = True,
                       num_chunks: int = 8, stream=None):
    """ep_dispatch_from_host.  h_x: bf16 CPU tensor [T, H] (pinned for overlap);
    d_x: CUDA staging tensor [T, H] (allocated when None).  num_chunks=0: the
    kernel reads h_x in place (h_x must be pinned; no staging, d_x stays
    None).  Returns (recv_x, recv_scale, recv_w, d_x)."""
    import torch

    cap, H = cfg.capacity, cfg.hidden
    dev = torch.device("cuda", torch.cuda.current_device())
    if d_x is None and num_chunks != 0:
        d_x = torch.empty(tuple(h_x.shape), dtype=torch.bfloat16, device=dev)
    if recv_x is None:
        dt = torch.uint8 if cfg.use_fp8_dispatch else torch.bfloat16
        recv_x = torch.empty((cap, H), dtype=dt, device=dev)
    if cfg.use_fp8_dispatch and recv_scale is None:
        recv_scale = torch.empty((cap, H // 128), dtype=torch.float32, device=dev)
    if want_weights and topk_weights is not None and recv_w is None:
        recv_w = torch.empty(cap, dtype=torch.float32, device=dev)
    st = ep_dispatch_from_host(cfg.c(), layout.c, _ptr(h_x), _ptr(d_x), _ptr(topk_weights),
                               _ptr(recv_x), _ptr(recv_scale), _ptr(recv_w), num_chunks,
                               _stream(stream))
    _check(st, "ep_dispatch_from_host")
    return recv_x, recv_scale, recv_w, d_x


def combine_to_host(cfg: Config, layout: Layout, expert_out, topk_weights=None, h_y=None,
                    d_y=None, num_chunks: int = 8, stream=None):
    """ep_combine_to_host.  Returns (h_y, d_y): h_y a pinned bf16 CPU tensor
    [T, H], readable once the stream has been synchronised.  num_chunks=0:
    the kernel writes h_y in place (h_y must be pinned; d_y stays None)."""
    import torch

    T, H = layout.num_tokens, cfg.hidden
    if h_y is None:
        h_y = torch.empty((T, H), dtype=torch.bfloat16).pin_memory()
    if d_y is None and num_chunks != 0:
        d_y = torch.empty((T, H), dtype=torch.bfloat16, device=expert_out.device)
    st = ep_combine_to_host(cfg.c(), layout.c, _ptr(expert_out), _ptr(topk_weights), _ptr(d_y),
                            _ptr(h_y), num_chunks, _stream(stream))
    _check(st, "ep_combine_to_host")
    return h_y, d_y


def check_error(layout: Layout, stream=None) -> int:
    return ep_check_error(layout.c, _stream(stream))


def dispatch_fp8(cfg: Config, layout: Layout, x=None, x_q=None, x_scale=None,
                 topk_weights=None, scale_col_major: bool = False, recv_q=None,
                 recv_scale=None, recv_w=None, want_weights: bool = True, stream=None):
    """ep_dispatch_fp8: quantise bf16 `x`, or copy pre-quantised `x_q` (uint8
    E4M3 bits [T, H]) with `x_scale` (fp32 [T, H/128]).  Returns (recv_q,
    recv_scale, recv_w); recv_scale is [cap, H/128], or [H/128, ld] when
    scale_col_major."""
    import torch

    cap, H = cfg.capacity, cfg.hidden
    dev = (x if x is not None else x_q).device
    if recv_q is None:
        recv_q = torch.empty((cap, H), dtype=torch.uint8, device=dev)
    if recv_scale is None:
        shape = (H // 128, ep_scale_ld(cfg.c())) if scale_col_major else (cap, H // 128)
        recv_scale = torch.empty(shape, dtype=torch.float32, device=dev)
    if want_weights and topk_weights is not None and recv_w is None:
        recv_w = torch.empty(cap, dtype=torch.float32, device=dev)
    st = ep_dispatch_fp8(cfg.c(), layout.c, _ptr(x), _ptr(x_q), _ptr(x_scale),
                         _ptr(topk_weights), _ptr(recv_q), _ptr(recv_scale),
                         scale_col_major, _ptr(recv_w), _stream(stream))
    _check(st, "ep_dispatch_fp8")
    return recv_q, recv_scale, recv_w


def combine_epilogue(cfg: Config, layout: Layout, expert_out, topk_weights=None,
                     bias0=None, bias1=None, recv_w=None, want_weights: bool = False,
                     y=None, stream=None):
    """ep_combine_epilogue.  Returns (y, combined_w or None)."""
    import torch

    T = layout.num_tokens
    dev = expert_out.device
    if y is None:
        y = torch.empty((T, cfg.hidden), dtype=torch.bfloat16, device=dev)
    cw = None
    if want_weights:
        cw = torch.empty((max(T, 1), cfg.num_topk), dtype=torch.float32, device=dev)
    st = ep_combine_epilogue(cfg.c(), layout.c, _ptr(expert_out), _ptr(topk_weights),
                             _ptr(bias0), _ptr(bias1), _ptr(recv_w), _ptr(y), _ptr(cw),
                             _stream(stream))
    _check(st, "ep_combine_epilogue")
    return y, (None if cw is None else cw[:T])


def dispatch_backward(cfg: Config, layout: Layout, grad_recv, grad_recv_w=None,
                      grad_x=None, stream=None):
    """ep_dispatch_backward.  Returns (grad_x bf16 [T, H], grad_w or None)."""
    import torch

    T = layout.num_tokens
    dev = grad_recv.device
    if grad_x is None:
        grad_x = torch.empty((T, cfg.hidden), dtype=torch.bfloat16, device=dev)
    gw = None
    if grad_recv_w is not None:
        gw = torch.empty((max(T, 1), cfg.num_topk), dtype=torch.float32, device=dev)
    st = ep_dispatch_backward(cfg.c(), layout.c, _ptr(grad_recv), _ptr(grad_recv_w),
                              _ptr(grad_x), _ptr(gw), _stream(stream))
    _check(st, "ep_dispatch_backward")
    return grad_x, (None if gw is None else gw[:T])


def combine_backward(cfg: Config, layout: Layout, dy, topk_weights=None, expert_out=None,
                     grad_expert_out=None, want_grad_w: bool = True, stream=None):
    """ep_combine_backward.  Returns (grad_expert_out bf16 [cap, H], grad_w or
    None); grad_w needs the forward expert rows `expert_out`."""
    import torch

    T = layout.num_tokens
    dev = dy.device
    if grad_expert_out is None:
        grad_expert_out = torch.empty((cfg.capacity, cfg.hidden), dtype=torch.bfloat16,
                                      device=dev)
    gw = None
    if want_grad_w and expert_out is not None:
        gw = torch.empty((max(T, 1), cfg.num_topk), dtype=torch.float32, device=dev)
    st = ep_combine_backward(cfg.c(), layout.c, _ptr(dy), _ptr(topk_weights),
                             _ptr(expert_out), _ptr(grad_expert_out), _ptr(gw),
                             _stream(stream))
    _check(st, "ep_combine_backward")
    return grad_expert_out, (None if gw is None else gw[:T])


# ---- non-expanded (destination-major) stage ------------------------------------

def dispatch_ranks(cfg: Config, layout: Layout, x, topk_idx, topk_weights=None,
                   stream=None):
    """ep_dispatch_ranks.  Returns (rank_x bf16 [rows_cap, H], rank_topk_idx
    int32 [rows_cap, K], rank_topk_w fp32 [rows_cap, K] or None)."""
    import torch

    n = ep_rank_rows_capacity(cfg.c())
    dev = x.device
    rank_x = torch.empty((max(n, 1), cfg.hidden), dtype=torch.bfloat16, device=dev)
    ridx = torch.empty((max(n, 1), cfg.num_topk), dtype=torch.int32, device=dev)
    rw = None
    if topk_weights is not None:
        rw = torch.empty((max(n, 1), cfg.num_topk), dtype=torch.float32, device=dev)
    st = ep_dispatch_ranks(cfg.c(), layout.c, _ptr(x), _ptr(topk_idx), _ptr(topk_weights),
                           _ptr(rank_x), _ptr(ridx), _ptr(rw), _stream(stream))
    _check(st, "ep_dispatch_ranks")
    return rank_x, ridx, rw


def expand(cfg: Config, layout: Layout, topk_idx, rank_x, rank_topk_w=None,
           recv_x=None, stream=None):
    """ep_expand.  Returns (recv_x bf16 [cap, H], recv_w or None)."""
    import torch

    dev = rank_x.device
    if recv_x is None:
        recv_x = torch.empty((cfg.capacity, cfg.hidden), dtype=torch.bfloat16, device=dev)
    rw = None
    if rank_topk_w is not None:
        rw = torch.empty(cfg.capacity, dtype=torch.float32, device=dev)
    st = ep_expand(cfg.c(), layout.c, _ptr(topk_idx), _ptr(rank_x), _ptr(rank_topk_w),
                   _ptr(recv_x), _ptr(rw), _stream(stream))
    _check(st, "ep_expand")
    return recv_x, rw


def reduce_ranks(cfg: Config, layout: Layout, topk_idx, expert_out, topk_weights=None,
                 stream=None):
    """ep_reduce_ranks.  Returns rank_y bf16 [rows_cap, H]."""
    import torch

    n = ep_rank_rows_capacity(cfg.c())
    rank_y = torch.empty((max(n, 1), cfg.hidden), dtype=torch.bfloat16,
                         device=expert_out.device)
    st = ep_reduce_ranks(cfg.c(), layout.c, _ptr(topk_idx), _ptr(expert_out),
                         _ptr(topk_weights), _ptr(rank_y), _stream(stream))
    _check(st, "ep_reduce_ranks")
    return rank_y


def combine_ranks(cfg: Config, layout: Layout, rank_y, y=None, stream=None):
    """ep_combine_ranks.  Returns y bf16 [T, H]."""
    import torch

    if y is None:
        y = torch.empty((layout.num_tokens, cfg.hidden), dtype=torch.bfloat16,
                        device=rank_y.device)
    st = ep_combine_ranks(cfg.c(), layout.c, _ptr(rank_y), _ptr(y), _stream(stream))
    _check(st, "ep_combine_ranks")
    return y


# ---- router gate -----------------------------------------------------------------
# The calls below sit in decode loops where a kernel takes a few microseconds:
# their ABI configs are built once, and a compiled extension (ep_torch_calls,
# csrc/torch_calls.cpp) checks the tensors and calls the library in one step.
# All tensors of a call are on the current GPU.  With `stream`, the caller lets
# that stream wait for the inputs, and whoever reads the outputs for it.

def _refuse(what: str):
    raise EpError(EP_ERR_INVALID_ARG, what)


def _done(status: int, what: str):
    if status < 0:
        _refuse(f"{what}: type, shape or place of a tensor")
    _check(status, f"ep_{what}")


class _LazyCalls:
    """ep_torch_calls, loaded with torch by the first call that needs it."""

    def __getattr__(self, name):
        global _calls
        import glob
        import importlib.machinery
        import importlib.metadata
        import importlib.util
        import sys

        import torch  # noqa: F401  (its libraries have to be there first)

        path = os.path.join(_PKG, "_lib", "ep_torch_calls.%s.torch%s.so" % (
            sys.implementation.cache_tag,
            importlib.metadata.version("torch").replace("+", ".")))
        if not os.path.exists(path):
            raise ImportError(
                f"{path} is missing (there: {glob.glob(path[:path.index('.cp')] + '*')}): "
                "build it with `python combine_get_layout_gb300/build_lib.py`")
        loader = importlib.machinery.ExtensionFileLoader("ep_torch_calls", path)
        mod = importlib.util.module_from_spec(
            importlib.util.spec_from_loader("ep_torch_calls", loader))
        loader.exec_module(mod)
        _calls = mod
        return getattr(mod, name)


_calls = _LazyCalls()


def _on_current_gpu(*tensors) -> bool:
    """Whether the tensors (None left out) are all on the current GPU, the one
    that the library launches on."""
    import torch

    try:
        gpu = torch._C._cuda_getDevice()
    except (AttributeError, RuntimeError):      # torch without CUDA, no GPU here
        return False
    return all(t is None or t.get_device() == gpu for t in tensors)


def _flat(t, dtype, shape) -> bool:
    """t is None, or a contiguous CUDA tensor of this type and shape."""
    return t is None or (t.dtype is dtype and t.is_cuda and t.is_contiguous()
                         and t.shape == shape)


def _outputs(stream, device, *wanted):
    """Uninitialised tensors, one for each (shape, type), for a call on this
    stream (None: the current one): made under it, so that what their memory
    was used for is over, and recorded on the current one, on which the
    caller may go on with them."""
    import torch

    here = None
    if stream is not None and device.type == "cuda":      # other places are refused later
        here = torch.cuda.current_stream(device)
    if here is None or here.cuda_stream == stream.cuda_stream:
        return tuple(torch.empty(shape, dtype=dtype, device=device) for shape, dtype in wanted)
    with torch.cuda.stream(stream):
        made = tuple(torch.empty(shape, dtype=dtype, device=device) for shape, dtype in wanted)
    for t in made:
        t.record_stream(here)
    return made


# Scratch memory of the eager calls, by (device, stream, host thread): calls
# of one thread on one stream run in order, so that they can share it.  A
# block that leaves the table goes back to its stream's memory, which later
# work of that stream alone takes it from.
_workspaces = {}
_workspaces_lock = _Lock()
_MOST_WORKSPACES = 32


def _workspace_of(t, stream, size: int):
    """At least `size` bytes on t's device for a call on this stream (None:
    the current one), made under it, so that nothing else that the memory was
    or will be used for overlaps.  Kept from call to call (asking the
    allocator each time costs more than the kernels of a small batch); where
    that stream is being captured, fresh memory that the graph owns."""
    import torch

    dev = t.get_device()
    if not _on_current_gpu(t):
        _refuse("route_balance: the logits are on another GPU than the current one")
    handle = torch._C._cuda_getCurrentRawStream(dev)
    if stream is not None and stream.cuda_stream != handle:
        with torch.cuda.stream(stream):
            return _workspace_of(t, None, size)
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(size, dtype=torch.uint8, device=t.device)
    key = dev, handle, _get_ident()
    got = _workspaces.get(key)
    if got is None or got.nbytes < size:
        got = torch.empty(max(size, 1 << 20), dtype=torch.uint8, device=t.device)
        with _workspaces_lock:
            _workspaces.pop(key, None)
            while len(_workspaces) >= _MOST_WORKSPACES:      # the first that was made
                del _workspaces[next(iter(_workspaces))]
            _workspaces[key] = got
    return got


class _AbiConfig:
    """A config that keeps its ABI struct and the struct's address.  Copies and
    pickles carry the fields alone: each object has a struct of its own."""

    def __reduce__(self):
        return type(self), tuple(getattr(self, f.name) for f in dataclasses.fields(self))

    def _same_numbers(self, c) -> bool:
        """Whether the struct holds the fields' whole numbers: ctypes drops the
        bits that do not fit."""
        return all(getattr(c, f.name) == getattr(self, f.name) for f in dataclasses.fields(self)
                   if f.type == "int")


@dataclasses.dataclass(frozen=True)
class RouterConfig(_AbiConfig):
    """Mirror of ep_router_config (see include/ep.h); the logits' type is
    taken from the tensors."""

    num_experts: int
    num_topk: int
    score: str = "softmax"          # or "sigmoid"
    num_groups: int = 1
    topk_groups: int = 1
    renormalize: bool = True
    route_scale: float = 1.0

    def __post_init__(self):
        if self.score not in ("softmax", "sigmoid"):
            _refuse(f"RouterConfig: score {self.score!r}")
        both = (EpRouterConfig * 2)(*(
            EpRouterConfig(self.num_experts, self.num_topk, int(self.score == "sigmoid"),
                           self.num_groups, self.topk_groups, int(self.renormalize), bf16,
                           self.route_scale) for bf16 in (0, 1)))
        if not self._same_numbers(both[0]):
            _refuse("RouterConfig: a number of over 32 bits")
        object.__setattr__(self, "_c", both)
        object.__setattr__(self, "_at", ctypes.addressof(both))

    def c(self, bf16: bool = False) -> EpRouterConfig:
        return self._c[int(bf16)]


def route(cfg: RouterConfig, logits, bias=None, token_mask=None, topk_idx=None,
          topk_weights=None, stream=None):
    """ep_route.  logits: fp32 or bf16 CUDA tensor [T, E], rows may be strided;
    bias: fp32 [E]; token_mask: uint8 or bool [T].  Returns (topk_idx int64
    [T, K], topk_weights fp32 [T, K])."""
    if topk_idx is None or topk_weights is None:
        import torch

        shape, dev = (logits.shape[0], cfg.num_topk), logits.device
        if topk_idx is None:
            topk_idx, = _outputs(stream, dev, (shape, torch.int64))
        if topk_weights is None:
            topk_weights, = _outputs(stream, dev, (shape, torch.float32))
    st = _calls.route(cfg._at, logits, bias, token_mask, topk_idx, topk_weights,
                      stream if stream is None else stream.cuda_stream)
    if st:
        _done(st, "route")
    return topk_idx, topk_weights


def route_balance(cfg: RouterConfig, logits, bias=None, token_mask=None, seq_start=None,
                  out=None, workspace=None, stream=None):
    """ep_route_balance.  seq_start: int32 [B + 1] CUDA tensor, or None for one
    sequence.  Returns (topk_idx, topk_weights, expert_count int32 [B, E],
    expert_prob fp32 [B, E], seq_tokens int32 [B + 2], loss fp32 [2]), which
    `out` may give; workspace: ep_route_workspace_bytes bytes (when None,
    memory kept for the calls of this thread on this stream)."""
    B = 1 if seq_start is None else seq_start.shape[0] - 1
    if out is None:
        import torch

        T, E, K, dev = logits.shape[0], cfg.num_experts, cfg.num_topk, logits.device
        out = _outputs(stream, dev, ((T, K), torch.int64), ((T, K), torch.float32),
                       ((B, E), torch.int32), ((B, E), torch.float32), ((B + 2,), torch.int32),
                       ((2,), torch.float32))
    size = _lib.ep_route_workspace_bytes(cfg._c[0], B)
    if size < 0 or not logits.is_cuda:
        _refuse("route_balance: config, number of sequences or place of the logits")
    if workspace is None:
        workspace = _workspace_of(logits, stream, size)
    idx, w, count, prob, tokens, loss = out
    st = _calls.route_balance(cfg._at, logits, bias, token_mask, seq_start, idx, w, count, prob,
                              tokens, loss, workspace, size,
                              stream if stream is None else stream.cuda_stream)
    if st:
        _done(st, "route_balance")
    return idx, w, count, prob, tokens, loss


def route_backward(cfg: RouterConfig, logits, topk_idx=None, grad_w=None, token_mask=None,
                   seq_start=None, expert_count=None, seq_tokens=None, grad_loss=None,
                   grad_logits=None, stream=None):
    """ep_route_backward.  grad_w: the gate weights' gradient (combine_backward
    returns it); expert_count, seq_tokens: route_balance's; grad_loss: fp32 [2]
    CUDA tensor.  Returns grad_logits [T, E] of the logits' type."""
    if grad_logits is None:
        grad_logits, = _outputs(stream, logits.device, (tuple(logits.shape), logits.dtype))
    st = _calls.route_backward(cfg._at, logits, topk_idx, grad_w, token_mask, seq_start,
                               expert_count, seq_tokens, grad_loss, grad_logits,
                               stream if stream is None else stream.cuda_stream)
    if st:
        _done(st, "route_backward")
    return grad_logits


# ---- experts' products with 4-bit weights ----------------------------------------

@dataclasses.dataclass(frozen=True)
class W4Config(_AbiConfig):
    """Mirror of ep_w4_config (see include/ep.h)."""

    num_experts: int
    in_features: int
    out_features: int
    group_size: int = 128
    x_fp8: bool = False
    gated: bool = False
    has_zeros: bool = False

    def __post_init__(self):
        c = EpW4Config(self.num_experts, self.in_features, self.out_features, self.group_size,
                       int(self.x_fp8), int(self.gated), int(self.has_zeros))
        sizes = ep_w4_codes_bytes(c), ep_w4_scales_bytes(c), ep_w4_zeros_bytes(c)
        if min(sizes) < 0 or not self._same_numbers(c):
            _refuse("W4Config")
        object.__setattr__(self, "_c", c)
        object.__setattr__(self, "_at", ctypes.addressof(c))
        object.__setattr__(self, "_width",
                           self.out_features // 2 if self.gated else self.out_features)

    def c(self) -> EpW4Config:
        return self._c

    @property
    def out_width(self) -> int:
        return self._width


def w4_pack(cfg: W4Config, codes, scales, zeros=None, stream=None):
    """ep_w4_pack.  codes: uint8 CUDA tensor [E, N, H / 2]; scales: bf16
    [E, N, H / group]; zeros: uint8, as the scales.  Returns the packed (codes
    int32 [E, tiles, blocks, 8, 32, 4], scales bf16 [E, tiles, groups, 64],
    zeros uint8 or None)."""
    import torch

    E, N, H, g = cfg.num_experts, cfg.out_features, cfg.in_features, cfg.group_size
    if not (_flat(codes, torch.uint8, (E, N, H // 2))
            and _flat(scales, torch.bfloat16, (E, N, H // g))
            and _flat(zeros, torch.uint8, (E, N, H // g)) and _on_current_gpu(codes, scales, zeros)):
        _refuse("w4_pack: type, shape or place of a tensor")
    tiles, blocks, dev = -(-cfg._width // (32 if cfg.gated else 64)), -(-H // 128), codes.device
    packed = (E, tiles, blocks * 128 // g, 64)
    pc, ps = _outputs(stream, dev, ((E, tiles, blocks, 8, 32, 4), torch.int32),
                      (packed, torch.bfloat16))
    pz, = _outputs(stream, dev, (packed, torch.uint8)) if cfg.has_zeros else (None,)
    st = ep_w4_pack(cfg._c, codes.data_ptr(), scales.data_ptr(), _ptr(zeros), pc.data_ptr(),
                    ps.data_ptr(), _ptr(pz), _stream(stream))
    _check(st, "ep_w4_pack")
    return pc, ps, pz


def expert_w4(cfg: W4Config, x, codes, scales, expert_start, expert_end, num_rows, zeros=None,
              x_scale=None, out=None, stream=None):
    """ep_expert_w4.  x: bf16 [cap, H], or uint8 (E4M3 bits) with x_scale fp32
    [cap, H / 128]; codes, scales, zeros: w4_pack's; expert_start, expert_end:
    a Layout's; num_rows: rows of all experts together at most (T * K).
    Returns out, bf16 [cap, N] ([cap, N / 2] when gated)."""
    if out is None:
        import torch

        out, = _outputs(stream, x.device, ((x.shape[0], cfg._width), torch.bfloat16))
    st = _calls.expert_w4(cfg._at, x, codes, scales, expert_start, expert_end, num_rows, zeros,
                          x_scale, out, stream if stream is None else stream.cuda_stream)
    if st:
        _done(st, "expert_w4")
    return out


# ---- experts' products with bf16 weights -------------------------------------------

@dataclasses.dataclass(frozen=True)
class ExpertConfig(_AbiConfig):
    """Mirror of ep_expert_config (see include/ep.h)."""

    num_experts: int
    in_features: int
    out_features: int
    x_fp8: bool = False
    gated: bool = False

    def __post_init__(self):
        c = EpExpertConfig(self.num_experts, self.in_features, self.out_features,
                           int(self.x_fp8), int(self.gated))
        # a call without rows checks the config alone
        at = 16
        if not self._same_numbers(c) or ep_expert_mm(c, 0, 0, None, None, at, at, at, None, None,
                                                     None) != EP_OK:
            _refuse("ExpertConfig")
        object.__setattr__(self, "_c", c)
        object.__setattr__(self, "_at", ctypes.addressof(c))
        object.__setattr__(self, "_width",
                           self.out_features // 2 if self.gated else self.out_features)

    def c(self) -> EpExpertConfig:
        return self._c

    @property
    def out_width(self) -> int:
        return self._width


def expert_mm(cfg: ExpertConfig, x, w, expert_start, expert_end, num_rows, x_scale=None, out=None,
              err=None, stream=None):
    """ep_expert_mm.  x: bf16 [cap, H], or uint8 (E4M3 bits) with x_scale fp32
    [cap, H / 128]; w: bf16 [E, N, H]; expert_start, expert_end: a Layout's;
    num_rows: rows of all experts together at most (T * K); err: a Layout's,
    or None.  Returns out, bf16 [cap, N] ([cap, N / 2] when gated)."""
    if out is None:
        import torch

        out, = _outputs(stream, x.device, ((x.shape[0], cfg._width), torch.bfloat16))
    st = _calls.expert_mm(cfg._at, x, w, expert_start, expert_end, num_rows, x_scale, out, err,
                          stream if stream is None else stream.cuda_stream)
    if st:
        _done(st, "expert_mm")
    return out


def expert_mm_backward(cfg: ExpertConfig, grad_out, expert_start, expert_end, num_rows, w=None,
                       x=None, x_scale=None, grad_x=None, grad_w=None, grad_w_dtype=None,
                       accumulate: bool = False, err=None, stream=None):
    """ep_expert_mm_backward.  grad_out: bf16 [cap, N].  With w (the forward
    call's) the gradient by the rows is computed, with x (and x_scale) the
    gradient by the weights: grad_w [E, N, H] of grad_w's type, or of
    grad_w_dtype (bf16 by default, or fp32) where it is None; accumulate: adds
    to grad_w (fp32).  Returns (grad_x bf16 [cap, H] or None, grad_w or
    None)."""
    if w is not None and grad_x is None:
        import torch

        grad_x, = _outputs(stream, grad_out.device,
                           ((grad_out.shape[0], cfg.in_features), torch.bfloat16))
    if x is not None and grad_w is None:
        import torch

        if accumulate:
            _refuse("expert_mm_backward: accumulate without grad_w")
        grad_w, = _outputs(stream, grad_out.device,
                           ((cfg.num_experts, cfg.out_features, cfg.in_features),
                            grad_w_dtype or torch.bfloat16))
    st = _calls.expert_mm_backward(cfg._at, grad_out, expert_start, expert_end, num_rows, w, x,
                                   x_scale, grad_x, grad_w, bool(accumulate), err,
                                   stream if stream is None else stream.cuda_stream)
    if st:
        _done(st, "expert_mm_backward")
    return grad_x, grad_w


# ---- gated activation with its input kept in 8 bits ----------------------------------

def act_save(h, expert_start, expert_end, num_rows, a=None, h_q=None, h_scale=None, stream=None):
    """ep_act_save.  h: bf16 [cap, 2 I], gate and up values side by side;
    expert_start (int32 [E + 1], or [E]), expert_end (int32 [E]), num_rows: as in expert_mm.
    Returns (a bf16 [cap, I], h_q uint8 (E4M3 bits) [cap, 2 I], h_scale fp32
    [cap, 2 ceil(I / 128)])."""
    if a is None or h_q is None or h_scale is None:
        import torch

        cap, width, dev = h.shape[0], h.shape[1] // 2, h.device
        if a is None:
            a, = _outputs(stream, dev, ((cap, width), torch.bfloat16))
        if h_q is None:
            h_q, = _outputs(stream, dev, ((cap, 2 * width), torch.uint8))
        if h_scale is None:
            h_scale, = _outputs(stream, dev, ((cap, 2 * -(-width // 128)), torch.float32))
    st = _calls.act_save(h, expert_start, expert_end, num_rows, a, h_q, h_scale,
                         stream if stream is None else stream.cuda_stream)
    if st:
        _done(st, "act_save")
    return a, h_q, h_scale


def act_backward(grad_a, h_q, h_scale, expert_start, expert_end, num_rows, grad_h=None, a=None,
                 want_a: bool = True, stream=None):
    """ep_act_backward.  grad_a: bf16 [cap, I]; h_q, h_scale: act_save's.
    Returns (grad_h bf16 [cap, 2 I], a bf16 [cap, I] or None)."""
    want_a = want_a or a is not None
    if grad_h is None or (a is None and want_a):
        import torch

        cap, width, dev = grad_a.shape[0], grad_a.shape[1], grad_a.device
        if grad_h is None:
            grad_h, = _outputs(stream, dev, ((cap, 2 * width), torch.bfloat16))
        if a is None and want_a:
            a, = _outputs(stream, dev, ((cap, width), torch.bfloat16))
    st = _calls.act_backward(grad_a, h_q, h_scale, expert_start, expert_end, num_rows, grad_h, a,
                             stream if stream is None else stream.cuda_stream)
    if st:
        _done(st, "act_backward")
    return grad_h, a
