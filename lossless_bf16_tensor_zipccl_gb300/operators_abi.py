"""The operator calls of ``include/zipccl.h`` (routing, plan, dispatch, combine,
AdamW step): records, argument types and pointer-level mirrors, without torch.
``operators`` has the same calls on tensors."""
from __future__ import annotations

import ctypes

from . import _check, load

__all__ = [
    "TYPE_F32", "TYPE_BF16", "TYPE_F16", "RouteOptions", "AdamWTensor", "AdamWOptions",
    "zipccl_moe_route", "zipccl_moe_route_backward", "zipccl_moe_plan_workspace_bytes", "zipccl_moe_plan",
    "zipccl_moe_dispatch", "zipccl_moe_dispatch_backward", "zipccl_moe_combine", "zipccl_moe_combine_backward",
    "zipccl_adamw_step",
]

TYPE_F32, TYPE_BF16, TYPE_F16 = range(3)


class RouteOptions(ctypes.Structure):
    _fields_ = [("top_k", ctypes.c_uint32), ("score", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float), ("groups", ctypes.c_uint32), ("groups_kept", ctypes.c_uint32),
                ("group_score", ctypes.c_int32)]


class AdamWTensor(ctypes.Structure):
    _fields_ = [("d_param", ctypes.c_void_p), ("d_grad", ctypes.c_void_p), ("d_exp_avg", ctypes.c_void_p),
                ("d_exp_avg_sq", ctypes.c_void_p), ("d_copy", ctypes.c_void_p), ("d_avg_scale", ctypes.c_void_p),
                ("d_sq_scale", ctypes.c_void_p), ("n", ctypes.c_uint64)]


class AdamWOptions(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("step", ctypes.c_uint64)]


def declare(L) -> None:
    """Argument types of the library's operator calls (used by ``load``)."""
    u64, u32, i32, vp = ctypes.c_uint64, ctypes.c_uint32, ctypes.c_int, ctypes.c_void_p
    ro = ctypes.POINTER(RouteOptions)
    L.zipccl_moe_route.argtypes = [vp, i32, u64, u64, u32, ro, vp, vp, vp, vp, vp]
    L.zipccl_moe_route_backward.argtypes = [vp, vp, i32, u64, u64, u32, ro, vp, vp, vp]
    L.zipccl_moe_plan_workspace_bytes.argtypes = [u64, u32, ctypes.POINTER(u64)]
    L.zipccl_moe_plan.argtypes = [vp, u64, u32, vp, vp, vp, vp, u64, vp]
    L.zipccl_moe_dispatch.argtypes = [vp, i32, u64, u64, u32, u64, vp, vp, vp]
    L.zipccl_moe_dispatch_backward.argtypes = [vp, i32, u64, u32, u64, vp, vp, vp]
    L.zipccl_moe_combine.argtypes = [vp, i32, u64, u32, u64, vp, vp, vp, vp, vp]
    L.zipccl_moe_combine_backward.argtypes = [vp, vp, i32, u64, u32, u64, vp, vp, vp, vp, vp]
    L.zipccl_adamw_step.argtypes = [ctypes.POINTER(AdamWTensor), u32, i32, i32, i32, ctypes.POINTER(AdamWOptions),
                                    vp, vp]
    for name in ("zipccl_moe_route", "zipccl_moe_route_backward", "zipccl_moe_plan_workspace_bytes",
                 "zipccl_moe_plan", "zipccl_moe_dispatch", "zipccl_moe_dispatch_backward", "zipccl_moe_combine",
                 "zipccl_moe_combine_backward", "zipccl_adamw_step"):
        getattr(L, name).restype = ctypes.c_int


# ------------------------------------------------------------------ C ABI mirrors
def zipccl_moe_route(d_logits: int, type: int, row_stride: int, tokens: int, experts: int, options: RouteOptions,
                     d_bias: int, d_mask: int, d_weights: int, d_ids: int, stream: int) -> int:
    return load().zipccl_moe_route(d_logits, type, row_stride, tokens, experts, options, d_bias, d_mask, d_weights,
                                   d_ids, stream)


def zipccl_moe_route_backward(d_grad_weights: int, d_logits: int, type: int, row_stride: int, tokens: int,
                              experts: int, options: RouteOptions, d_ids: int, d_grad_logits: int,
                              stream: int) -> int:
    return load().zipccl_moe_route_backward(d_grad_weights, d_logits, type, row_stride, tokens, experts, options,
                                            d_ids, d_grad_logits, stream)


def zipccl_moe_plan_workspace_bytes(pairs: int, experts: int) -> int:
    out = ctypes.c_uint64()
    _check(load().zipccl_moe_plan_workspace_bytes(int(pairs), int(experts), ctypes.byref(out)),
           "zipccl_moe_plan_workspace_bytes")
    return int(out.value)


def zipccl_moe_plan(d_ids: int, pairs: int, experts: int, d_counts: int, d_offsets: int, d_slots: int, d_ws: int,
                    ws_bytes: int, stream: int) -> int:
    return load().zipccl_moe_plan(d_ids, pairs, experts, d_counts, d_offsets, d_slots, d_ws, ws_bytes, stream)


def zipccl_moe_dispatch(d_x: int, type: int, row_stride: int, tokens: int, top_k: int, hidden: int, d_slots: int,
                        d_rows: int, stream: int) -> int:
    return load().zipccl_moe_dispatch(d_x, type, row_stride, tokens, top_k, hidden, d_slots, d_rows, stream)


def zipccl_moe_dispatch_backward(d_grad_rows: int, type: int, tokens: int, top_k: int, hidden: int, d_slots: int,
                                 d_grad_x: int, stream: int) -> int:
    return load().zipccl_moe_dispatch_backward(d_grad_rows, type, tokens, top_k, hidden, d_slots, d_grad_x, stream)


def zipccl_moe_combine(d_rows: int, type: int, tokens: int, top_k: int, hidden: int, d_slots: int, d_weights: int,
                       d_residual: int, d_y: int, stream: int) -> int:
    return load().zipccl_moe_combine(d_rows, type, tokens, top_k, hidden, d_slots, d_weights, d_residual, d_y, stream)


def zipccl_moe_combine_backward(d_grad_y: int, d_rows: int, type: int, tokens: int, top_k: int, hidden: int,
                                d_slots: int, d_weights: int, d_grad_rows: int, d_grad_weights: int,
                                stream: int) -> int:
    return load().zipccl_moe_combine_backward(d_grad_y, d_rows, type, tokens, top_k, hidden, d_slots, d_weights,
                                              d_grad_rows, d_grad_weights, stream)


def zipccl_adamw_step(tensors, n_tensors: int, param_type: int, grad_type: int, state_bits: int,
                      options: AdamWOptions, d_grad_scale: int, stream: int) -> int:
    """tensors: a ctypes array of at least n_tensors AdamWTensor records."""
    return load().zipccl_adamw_step(tensors, n_tensors, param_type, grad_type, state_bits, options, d_grad_scale,
                                    stream)
