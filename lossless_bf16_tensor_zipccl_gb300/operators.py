"""Operators around the compressed exchange, on torch tensors: routing to
experts, the chunk plan, dispatch and combine with their gradients, and the
AdamW step over many tensors.

They make and use what ``compress`` packs: a router's choice and ``moe_plan``
give the per-expert chunks (``plan.counts * hidden`` is ``chunk_elems``),
``moe_dispatch`` fills them, ``moe_combine`` brings the rows back, and
``adamw_step`` takes the gradient shard that ``decompress_reduce`` returns.

They are the ``zipccl_moe_*`` and ``zipccl_adamw_step`` calls of
``include/zipccl.h`` (which states each formula) on CUDA tensors.  Like the
rest of the package they run on the current stream unless ``stream`` is given,
allocate their results unless these are passed in, raise ``TypeError`` /
``ValueError`` for tensors they cannot take and ``ZipcclError`` for what the
library refuses.
"""
from __future__ import annotations

from array import array
from functools import lru_cache
from typing import NamedTuple

import torch

from . import _check, _keep
from .operators_abi import (TYPE_BF16, TYPE_F16, TYPE_F32, AdamWOptions, AdamWTensor, RouteOptions, zipccl_adamw_step,
                            zipccl_moe_combine, zipccl_moe_combine_backward, zipccl_moe_dispatch,
                            zipccl_moe_dispatch_backward, zipccl_moe_plan, zipccl_moe_plan_workspace_bytes,
                            zipccl_moe_route, zipccl_moe_route_backward)

__all__ = ["ADAMW_BLOCK", "MoePlan", "moe_route", "moe_route_backward", "moe_plan", "moe_dispatch",
           "moe_dispatch_backward", "moe_combine", "moe_combine_backward", "adamw_step", "adamw_state"]

ADAMW_BLOCK = 256  # values that share one scale of an 8-bit state

_TYPES = {torch.float32: TYPE_F32, torch.bfloat16: TYPE_BF16, torch.float16: TYPE_F16}
_SCORES = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORES = {"max": 0, "top2": 1}


class MoePlan(NamedTuple):
    """Chunk layout of routed pairs: rows of each expert's chunk, first row of
    each (and the rows in all), and the row of every pair (-1 - row where the
    pair is dropped)."""
    counts: torch.Tensor
    offsets: torch.Tensor
    slots: torch.Tensor


# The stream's handle without building a Stream object: 0.1 us instead of 2.9
# of the 8 us that a small call takes in all (measured on the Arm host).
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream, t) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _current_raw_stream is not None:
        return _current_raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _type(t, what: str) -> int:
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what}: expected float32, bfloat16 or float16, got {t.dtype}")
    return code


def _plain(t, dtype, shape, what: str):
    """A contiguous CUDA tensor of this type and shape."""
    if t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous CUDA tensor")
    return t


def _rows(t, what: str) -> int:
    """Row stride of a [tokens, values] CUDA tensor whose rows are contiguous."""
    if t.dim() != 2:
        raise ValueError(f"{what}: expected two dimensions, got {tuple(t.shape)}")
    n, m = t.shape
    s0, s1 = t.stride()
    if not t.is_cuda or (s1 != 1 and m > 1):
        raise ValueError(f"{what}: expected a CUDA tensor with contiguous rows")
    return s0 if n > 1 else max(s0, m)


def _result(t, shape, dtype, like, what: str, stream):
    if t is not None:
        return _plain(t, dtype, shape, what)
    t = torch.empty(shape, dtype=dtype, device=like.device)
    return t if stream is None else _keep(t, stream)


@lru_cache(maxsize=64)
def _route_options(top_k, score, renormalize, scale, groups, groups_kept, group_score) -> RouteOptions:
    if score not in _SCORES:
        raise ValueError(f"score: expected one of {sorted(_SCORES)}, got {score!r}")
    if group_score not in _GROUP_SCORES:
        raise ValueError(f"group_score: expected one of {sorted(_GROUP_SCORES)}, got {group_score!r}")
    if min(top_k, groups, groups_kept) < 1:
        raise ValueError("top_k, groups and groups_kept are at least 1")
    return RouteOptions(top_k, _SCORES[score], bool(renormalize), scale, groups, groups_kept,
                        _GROUP_SCORES[group_score])


def moe_route(logits, top_k: int, *, score: str = "softmax", bias=None, groups: int = 1, groups_kept: int = 1,
              group_score: str = "max", renormalize: bool = True, scale: float = 1.0, mask=None, weights=None,
              ids=None, stream=None):
    """Experts of every token: (weights [tokens, top_k] float32, ids [tokens,
    top_k] int32, best first) from logits [tokens, experts].  ``score`` is
    "softmax" or "sigmoid"; ``bias`` (float32 [experts]) shifts the choice
    only; with ``groups`` > 1 each token chooses within its ``groups_kept`` best
    groups, ranked by their "max" or "top2" sum; ``mask`` (bool or uint8
    [tokens]) leaves tokens out: ids -1, weights 0 (see zipccl_moe_route)."""
    opt = _route_options(top_k, score, renormalize, scale, groups, groups_kept, group_score)
    kind, stride = _type(logits, "logits"), _rows(logits, "logits")
    tokens, experts = logits.shape
    if bias is not None:
        _plain(bias, torch.float32, (experts,), "bias")
    if mask is not None:
        _plain(mask, mask.dtype if mask.dtype in (torch.bool, torch.uint8) else torch.bool, (tokens,), "mask")
    weights = _result(weights, (tokens, top_k), torch.float32, logits, "weights", stream)
    ids = _result(ids, (tokens, top_k), torch.int32, logits, "ids", stream)
    st = zipccl_moe_route(logits.data_ptr(), kind, stride, tokens, experts, opt,
                          None if bias is None else bias.data_ptr(), None if mask is None else mask.data_ptr(),
                          weights.data_ptr(), ids.data_ptr(), _raw_stream(stream, logits))
    if st:
        _check(st, "zipccl_moe_route")
    return weights, ids


def moe_route_backward(grad_weights, logits, ids, *, score: str = "softmax", renormalize: bool = True,
                       scale: float = 1.0, grad_logits=None, stream=None):
    """Gradient of ``moe_route``'s weights by the logits (of their type), for
    the ids it returned and the same score, renormalize and scale."""
    tokens, experts = logits.shape
    top_k = ids.shape[-1]
    opt = _route_options(top_k, score, renormalize, scale, 1, 1, "max")
    kind, stride = _type(logits, "logits"), _rows(logits, "logits")
    _plain(ids, torch.int32, (tokens, top_k), "ids")
    _plain(grad_weights, torch.float32, (tokens, top_k), "grad_weights")
    grad_logits = _result(grad_logits, (tokens, experts), logits.dtype, logits, "grad_logits", stream)
    st = zipccl_moe_route_backward(grad_weights.data_ptr(), logits.data_ptr(), kind, stride, tokens, experts, opt,
                                   ids.data_ptr(), grad_logits.data_ptr(), _raw_stream(stream, logits))
    if st:
        _check(st, "zipccl_moe_route_backward")
    return grad_logits


def moe_plan(ids, n_experts: int, *, counts=None, offsets=None, slots=None, ws=None, stream=None) -> MoePlan:
    """Chunk layout of the pairs in ids [tokens, top_k] (int32; outside
    0..n_experts-1: dropped): counts [n_experts], offsets [n_experts + 1] and
    slots like ids, all int32 (see zipccl_moe_plan).  ``plan.counts * hidden``
    is the chunk_elems of the dispatched rows."""
    _plain(ids, torch.int32, ids.shape, "ids")
    pairs = ids.numel()
    need = zipccl_moe_plan_workspace_bytes(pairs, n_experts)
    counts = _result(counts, (n_experts,), torch.int32, ids, "counts", stream)
    offsets = _result(offsets, (n_experts + 1,), torch.int32, ids, "offsets", stream)
    slots = _result(slots, ids.shape, torch.int32, ids, "slots", stream)
    if need and (ws is None or ws.numel() * ws.element_size() < need):
        ws = _keep(torch.empty(need, dtype=torch.uint8, device=ids.device), stream)
    st = zipccl_moe_plan(ids.data_ptr(), pairs, n_experts, counts.data_ptr(), offsets.data_ptr(), slots.data_ptr(),
                         ws.data_ptr() if need else None, ws.numel() * ws.element_size() if need else 0,
                         _raw_stream(stream, ids))
    if st:
        _check(st, "zipccl_moe_plan")
    return MoePlan(counts, offsets, slots)


def moe_dispatch(x, slots, *, out=None, stream=None):
    """Rows of the experts' chunks, [tokens * top_k, hidden]: x[token] at each
    of its pairs' slots (``plan.slots``, [tokens, top_k]); rows of dropped
    pairs are zeros.  x [tokens, hidden] may have any row stride."""
    kind, stride = _type(x, "x"), _rows(x, "x")
    tokens, hidden = x.shape
    top_k = slots.shape[-1]
    _plain(slots, torch.int32, (tokens, top_k), "slots")
    out = _result(out, (tokens * top_k, hidden), x.dtype, x, "out", stream)
    st = zipccl_moe_dispatch(x.data_ptr(), kind, stride, tokens, top_k, hidden, slots.data_ptr(), out.data_ptr(),
                             _raw_stream(stream, x))
    if st:
        _check(st, "zipccl_moe_dispatch")
    return out


def _pairs(rows, slots, what: str):
    kind = _type(rows, what)
    tokens, top_k = slots.shape
    _plain(slots, torch.int32, (tokens, top_k), "slots")
    if rows.dim() != 2:
        raise ValueError(f"{what}: expected two dimensions, got {tuple(rows.shape)}")
    hidden = rows.shape[1]
    _plain(rows, rows.dtype, (tokens * top_k, hidden), what)
    return kind, tokens, top_k, hidden


def moe_dispatch_backward(grad_rows, slots, *, out=None, stream=None):
    """Gradient of ``moe_dispatch`` by x: the sum of each token's rows of
    grad_rows, [tokens, hidden]."""
    kind, tokens, top_k, hidden = _pairs(grad_rows, slots, "grad_rows")
    out = _result(out, (tokens, hidden), grad_rows.dtype, grad_rows, "out", stream)
    st = zipccl_moe_dispatch_backward(grad_rows.data_ptr(), kind, tokens, top_k, hidden, slots.data_ptr(),
                                      out.data_ptr(), _raw_stream(stream, grad_rows))
    if st:
        _check(st, "zipccl_moe_dispatch_backward")
    return out


def moe_combine(rows, slots, weights=None, *, residual=None, out=None, stream=None):
    """The experts' rows [tokens * top_k, hidden] back at their tokens:
    residual + sum of weight * row over each token's pairs, [tokens, hidden].
    ``weights`` is float32 [tokens, top_k] (None: 1)."""
    kind, tokens, top_k, hidden = _pairs(rows, slots, "rows")
    if weights is not None:
        _plain(weights, torch.float32, (tokens, top_k), "weights")
    if residual is not None:
        _plain(residual, rows.dtype, (tokens, hidden), "residual")
    out = _result(out, (tokens, hidden), rows.dtype, rows, "out", stream)
    st = zipccl_moe_combine(rows.data_ptr(), kind, tokens, top_k, hidden, slots.data_ptr(),
                            None if weights is None else weights.data_ptr(),
                            None if residual is None else residual.data_ptr(), out.data_ptr(), _raw_stream(stream, rows))
    if st:
        _check(st, "zipccl_moe_combine")
    return out


def moe_combine_backward(grad_out, rows, slots, weights=None, *, grad_rows=None, grad_weights=None, stream=None):
    """Gradients of ``moe_combine``: (grad_rows, of rows' type and shape, zeros
    for dropped pairs; grad_weights, float32 [tokens, top_k]).  The residual's
    gradient is grad_out itself."""
    kind, tokens, top_k, hidden = _pairs(rows, slots, "rows")
    _plain(grad_out, rows.dtype, (tokens, hidden), "grad_out")
    if weights is not None:
        _plain(weights, torch.float32, (tokens, top_k), "weights")
    grad_rows = _result(grad_rows, rows.shape, rows.dtype, rows, "grad_rows", stream)
    grad_weights = _result(grad_weights, (tokens, top_k), torch.float32, rows, "grad_weights", stream)
    st = zipccl_moe_combine_backward(grad_out.data_ptr(), rows.data_ptr(), kind, tokens, top_k, hidden,
                                     slots.data_ptr(), None if weights is None else weights.data_ptr(),
                                     grad_rows.data_ptr(), grad_weights.data_ptr(), _raw_stream(stream, rows))
    if st:
        _check(st, "zipccl_moe_combine_backward")
    return grad_rows, grad_weights


def adamw_state(param, bits: int = 32):
    """Zero states of one parameter for ``adamw_step``: (exp_avg, exp_avg_sq)
    with 32 bits; with 8, (exp_avg, exp_avg_sq, avg_scale, sq_scale)."""
    n, dev = param.numel(), param.device
    if bits == 32:
        return tuple(torch.zeros(param.shape, dtype=torch.float32, device=dev) for _ in range(2))
    if bits != 8:
        raise ValueError("states are held in 32 or 8 bits")
    codes = tuple(torch.zeros(param.shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2))
    return codes + tuple(torch.zeros(-(-n // ADAMW_BLOCK), dtype=torch.float32, device=dev) for _ in range(2))


def _column(tensors, sizes, dtype, what: str):
    """The addresses of one list of tensors, checked against the parameters'."""
    if len(tensors) != len(sizes):
        raise ValueError(f"{what}: expected {len(sizes)} tensors, got {len(tensors)}")
    found = []
    for t, n in zip(tensors, sizes):
        if t.dtype != dtype:
            raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{what}: expected contiguous CUDA tensors")
        if t.numel() != n:
            raise ValueError(f"{what}: expected {n} values, got {t.numel()}")
        found.append(t.data_ptr())
    return found


def adamw_step(params, grads, exp_avgs, exp_avg_sqs, *, step: int, lr: float, betas=(0.9, 0.999), eps: float = 1e-8,
               weight_decay: float = 0.01, scales=None, copies=None, grad_scale=None, stream=None) -> None:
    """One AdamW step over lists of tensors, in place (see zipccl_adamw_step).
    params and grads: float32 or bfloat16, one type for each list; exp_avgs and
    exp_avg_sqs: float32, or float8_e4m3fn with ``scales`` = (avg_scales,
    sq_scales), lists of float32 [ceil(n / 256)] (``adamw_state`` makes either;
    exp_avg_sqs then hold the root of the second moment).  ``copies``: bfloat16
    tensors that receive the new parameters; ``grad_scale``: a float32 CUDA
    scalar that every gradient is multiplied with."""
    n = len(params)
    if n == 0:
        return
    for what, tensors in (("params", params), ("grads", grads)):
        if len(tensors) != n or tensors[0].dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"{what}: expected {n} float32 or bfloat16 tensors")
    bits = 32 if scales is None else 8
    state = torch.float32 if bits == 32 else torch.float8_e4m3fn
    sizes = [p.numel() for p in params]
    none = [0] * n
    columns = [_column(params, sizes, params[0].dtype, "params"), _column(grads, sizes, grads[0].dtype, "grads"),
               _column(exp_avgs, sizes, state, "exp_avgs"), _column(exp_avg_sqs, sizes, state, "exp_avg_sqs"),
               none if copies is None else _column(copies, sizes, torch.bfloat16, "copies"), none, none, sizes]
    if bits == 8:
        blocks = [-(-m // ADAMW_BLOCK) for m in sizes]
        columns[5:7] = (_column(s, blocks, torch.float32, "scales") for s in scales)
    if grad_scale is not None:
        _plain(grad_scale, torch.float32, grad_scale.shape, "grad_scale")
        if grad_scale.numel() != 1:
            raise ValueError("grad_scale: expected one value")
    # the records' eight 64-bit fields, tensor by tensor
    words = array("Q", [0]) * (8 * n)
    for i, column in enumerate(columns):
        words[i::8] = array("Q", column)
    opt = AdamWOptions(lr, betas[0], betas[1], eps, weight_decay, step)
    _check(zipccl_adamw_step((AdamWTensor * n).from_buffer(words), n, _TYPES[params[0].dtype], _TYPES[grads[0].dtype],
                             bits, opt, None if grad_scale is None else grad_scale.data_ptr(),
                             _raw_stream(stream, params[0])), "zipccl_adamw_step")
