"""Operators around the compressed exchange, on torch tensors: routing to
experts, the chunk plan, dispatch and combine with their gradients, the experts'
products in 8 bits with theirs, the layer for a few tokens, and the AdamW step
over many tensors.

They make and use what ``compress`` packs: a router's choice and ``moe_plan``
give the per-expert chunks (``plan.counts * hidden`` is ``chunk_elems``),
``moe_dispatch`` fills them, ``moe_combine`` brings the rows back, and
``adamw_step`` takes the gradient shard that ``decompress_reduce`` returns.

They are the ``zipccl_moe_*`` and ``zipccl_adamw_step`` calls of
``include/zipccl.h`` (which states each formula) on CUDA tensors.  Like the
rest of the package they run on the current stream unless ``stream`` is given,
allocate their results unless these are passed in, raise ``TypeError`` /
``ValueError`` for tensors they cannot take and ``ZipcclError`` for what the
library refuses.  Autograd does not go through them: results carry no gradient
(a call that it would expect to go through warns), the ``_backward`` calls
compute gradients, and what is written in place counts as changed.  Results
allocated for another ``stream`` may be read by the current one after it has
waited for that stream.
"""
from __future__ import annotations

import importlib.util
from typing import NamedTuple

import torch

from . import _build, _check, load

__all__ = ["ADAMW_BLOCK", "MoePlan", "moe_route", "moe_route_backward", "moe_plan", "moe_dispatch",
           "moe_dispatch_backward", "moe_combine", "moe_combine_backward", "adamw_step", "adamw_state", "FP8_BLOCK",
           "Fp8Blocks", "moe_quantize", "moe_quantize_columns", "moe_quantize_weights", "moe_matmul",
           "moe_matmul_backward", "moe_matmul_backward_weights", "moe_status", "moe_layer"]

ADAMW_BLOCK = 256  # values that share one scale of an 8-bit state
FP8_BLOCK = 128    # values, rows or both that share one scale of 8-bit operands

_SCORES = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORES = {"max": 0, "top2": 1}
_ACTIVATIONS = {"silu": 0, "gelu": 1, "relu": 2}
_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_FORWARD, _BACKWARD, _WEIGHTS = range(3)


def _load_native():
    """The extension that checks tensors, allocates results and makes the call."""
    load()
    spec = importlib.util.spec_from_file_location("_zipccl_torch", _build.torch_extension())
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


_native = _load_native()


class MoePlan(NamedTuple):
    """Chunk layout of routed pairs: rows of each expert's chunk, first row of
    each (and the rows in all), and the row of every pair (-1 - row where the
    pair is dropped)."""
    counts: torch.Tensor
    offsets: torch.Tensor
    slots: torch.Tensor


class Fp8Blocks(NamedTuple):
    """8-bit values: codes (float8_e4m3fn, rows a multiple of 16 bytes apart)
    times a power of two for each block of 128 (scales, float8_e8m0fnu,
    contiguous)."""
    codes: torch.Tensor
    scales: torch.Tensor


def _choice(options, name, value):
    try:
        return options[value]
    except KeyError:
        raise ValueError(f"{name}: expected one of {sorted(options)}, got {value!r}") from None


def _handle(stream):
    return None if stream is None else stream.cuda_stream


def _done(result, what: str):
    if type(result) is int:
        _check(result, what)
    return result


def moe_route(logits, top_k: int, *, score: str = "softmax", bias=None, groups: int = 1, groups_kept: int = 1,
              group_score: str = "max", renormalize: bool = True, scale: float = 1.0, mask=None, weights=None,
              ids=None, stream=None):
    """Experts of every token: (weights [tokens, top_k] float32, ids [tokens,
    top_k] int32, best first) from logits [tokens, experts].  ``score`` is
    "softmax" or "sigmoid"; ``bias`` (float32 [experts]) shifts the choice
    only; with ``groups`` > 1 each token chooses within its ``groups_kept`` best
    groups, ranked by their "max" or "top2" sum; ``mask`` (bool or uint8
    [tokens]) leaves tokens out: ids -1, weights 0 (see zipccl_moe_route)."""
    return _done(_native.route(logits, top_k, _choice(_SCORES, "score", score), renormalize, scale, groups, groups_kept,
                               _choice(_GROUP_SCORES, "group_score", group_score), bias, mask, weights, ids,
                               _handle(stream)), "zipccl_moe_route")


def moe_route_backward(grad_weights, logits, ids, *, score: str = "softmax", renormalize: bool = True,
                       scale: float = 1.0, grad_logits=None, stream=None):
    """Gradient of ``moe_route``'s weights by the logits (of their type), for
    the ids it returned and the same score, renormalize and scale."""
    return _done(_native.route_backward(grad_weights, logits, ids, _choice(_SCORES, "score", score), renormalize, scale,
                                        grad_logits, _handle(stream)), "zipccl_moe_route_backward")


def moe_plan(ids, n_experts: int, *, counts=None, offsets=None, slots=None, ws=None, stream=None) -> MoePlan:
    """Chunk layout of the pairs in ids [tokens, top_k] (int32; outside
    0..n_experts-1: dropped): counts [n_experts], offsets [n_experts + 1] and
    slots like ids, all int32 (see zipccl_moe_plan).  ``plan.counts * hidden``
    is the chunk_elems of the dispatched rows."""
    return MoePlan(*_done(_native.plan(ids, n_experts, counts, offsets, slots, ws, _handle(stream)),
                          "zipccl_moe_plan"))


def moe_dispatch(x, slots, *, out=None, stream=None):
    """Rows of the experts' chunks, [tokens * top_k, hidden]: x[token] at each
    of its pairs' slots (``plan.slots``, [tokens, top_k]); rows of dropped
    pairs are zeros.  x [tokens, hidden] may have any row stride."""
    return _done(_native.dispatch(x, slots, out, _handle(stream)), "zipccl_moe_dispatch")


def moe_dispatch_backward(grad_rows, slots, *, out=None, stream=None):
    """Gradient of ``moe_dispatch`` by x: the sum of each token's rows of
    grad_rows, [tokens, hidden]."""
    return _done(_native.dispatch_backward(grad_rows, slots, out, _handle(stream)), "zipccl_moe_dispatch_backward")


def moe_combine(rows, slots, weights=None, *, residual=None, out=None, stream=None):
    """The experts' rows [tokens * top_k, hidden] back at their tokens:
    residual + sum of weight * row over each token's pairs, [tokens, hidden].
    ``weights`` is float32 [tokens, top_k] (None: 1)."""
    return _done(_native.combine(rows, slots, weights, residual, out, _handle(stream)), "zipccl_moe_combine")


def moe_combine_backward(grad_out, rows, slots, weights=None, *, grad_rows=None, grad_weights=None, stream=None):
    """Gradients of ``moe_combine``: (grad_rows, of rows' type and shape, zeros
    for dropped pairs; grad_weights, float32 [tokens, top_k]).  The residual's
    gradient is grad_out itself."""
    return _done(_native.combine_backward(grad_out, rows, slots, weights, grad_rows, grad_weights, _handle(stream)),
                 "zipccl_moe_combine_backward")


def moe_quantize(rows, *, out=None, stream=None) -> Fp8Blocks:
    """rows [n, cols] in 8 bits, blocks of 128 values along a row (see
    zipccl_moe_quantize): codes [n, cols], scales [n, ceil(cols / 128)].  Rows
    may have any stride.  The operand of ``moe_matmul`` and, for gradients, of
    ``moe_matmul_backward``."""
    return Fp8Blocks(*_done(_native.quantize(rows, out, _handle(stream)), "zipccl_moe_quantize"))


def moe_quantize_columns(rows, offsets=None, *, by_rows: bool = False, out=None, rows_out=None, stream=None):
    """rows [n, cols] in 8 bits, blocks of 128 rows of a chunk down a column:
    codes [n, cols], scales [n // 128 + experts, cols].  ``offsets`` is
    ``plan.offsets`` (None: all rows are one chunk).  With ``by_rows`` what
    ``moe_quantize`` gives too, from the same reading: (by rows, by columns).
    Both operands of ``moe_matmul_backward_weights``."""
    made = _done(_native.quantize_columns(rows, offsets, by_rows, out, rows_out, _handle(stream)),
                 "zipccl_moe_quantize_columns")
    return (Fp8Blocks(*made[0]), Fp8Blocks(*made[1])) if by_rows else Fp8Blocks(*made)


def moe_quantize_weights(weights, *, out=None, stream=None) -> Fp8Blocks:
    """The experts' matrices [experts, outer, inner] (or one, [outer, inner]) in
    8 bits, blocks of 128 x 128: forward and backward read the same codes."""
    return Fp8Blocks(*_done(_native.quantize_weights(weights, out, _handle(stream)), "zipccl_moe_quantize_weights"))


def _matmul(form, a, b, offsets, dtype, out, stream):
    try:
        type_ = _TYPES[dtype]
    except KeyError:
        raise TypeError(f"dtype: expected float32, bfloat16 or float16, got {dtype}") from None
    return _done(_native.matmul(form, a, b, offsets, type_, out, _handle(stream)), "zipccl_moe_matmul")


def moe_matmul(rows, weights, offsets=None, *, dtype=torch.bfloat16, out=None, stream=None):
    """Every row times its expert's matrix: out[m] = weights[e] @ rows[m] for the
    rows of chunk e, [n, outer]; rows behind the last chunk become zeros, as does
    everything where the matrices have no columns.
    ``rows`` from ``moe_quantize``, ``weights`` from ``moe_quantize_weights``;
    without ``offsets`` one matrix [outer, inner] for all rows."""
    return _matmul(_FORWARD, rows, weights, offsets, dtype, out, stream)


def moe_matmul_backward(grad_rows, weights, offsets=None, *, dtype=torch.bfloat16, out=None, stream=None):
    """Gradient of ``moe_matmul`` by the rows, [n, inner], from the result's
    gradient in 8 bits by rows (``moe_quantize``)."""
    return _matmul(_BACKWARD, grad_rows, weights, offsets, dtype, out, stream)


def moe_matmul_backward_weights(grad_columns, columns, offsets=None, *, dtype=torch.bfloat16, out=None, stream=None):
    """Gradient of ``moe_matmul`` by the weights, [experts, outer, inner] (one
    matrix without ``offsets``), from the result's gradient and the rows, both
    by columns of the same chunks (``moe_quantize_columns``)."""
    return _matmul(_WEIGHTS, grad_columns, columns, offsets, dtype, out, stream)


def moe_status(stream=None) -> None:
    """Raises ``ZipcclError`` if a wait inside a ``moe_matmul`` or ``moe_layer``
    call (or a gradient's) on the current device has run out since ``moe_status``
    was last called (synchronizes)."""
    handle = torch.cuda.current_stream().cuda_stream if stream is None else stream.cuda_stream
    _check(load().zipccl_moe_status(handle), "zipccl_moe_status")


def moe_layer(x, router, up, down, top_k: int, *, score: str = "softmax", bias=None, groups: int = 1,
              groups_kept: int = 1, group_score: str = "max", renormalize: bool = True, scale: float = 1.0, mask=None,
              activation: str = "silu", residual=None, out=None, weights=None, ids=None, ws=None, stream=None):
    """A whole layer for up to 32 tokens, in two kernels: (y [tokens, hidden],
    weights and ids [tokens, top_k] as ``moe_route`` gives them for the logits
    x @ router.T; see zipccl_moe_layer).  ``router`` is [experts, hidden], of x's
    type or float32; ``up`` [experts, inner or 2 * inner, hidden] (twice as many
    rows: the first half is the gate's) and ``down`` [experts, hidden, inner], both
    of x's type or both ``Fp8Blocks`` from ``moe_quantize_weights``;
    ``activation`` "silu", "gelu" or "relu".  x may have any row stride, 0
    (expanded) included.  For more tokens: route, plan, dispatch, ``moe_matmul``, combine."""
    return _done(_native.layer(x, router, up, down, top_k, _choice(_SCORES, "score", score), renormalize, scale, groups,
                               groups_kept, _choice(_GROUP_SCORES, "group_score", group_score), bias, mask,
                               _choice(_ACTIVATIONS, "activation", activation), residual, out, weights, ids, ws,
                               _handle(stream)), "zipccl_moe_layer")


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


def adamw_step(params, grads, exp_avgs, exp_avg_sqs, *, step: int, lr: float, betas=(0.9, 0.999), eps: float = 1e-8,
               weight_decay: float = 0.01, scales=None, copies=None, grad_scale=None, stream=None) -> None:
    """One AdamW step over lists (or iterators) of tensors, in place (see zipccl_adamw_step).
    params and grads: float32 or bfloat16, one type for each list; exp_avgs and
    exp_avg_sqs: float32, or float8_e4m3fn with ``scales`` = (avg_scales,
    sq_scales), lists of float32 [ceil(n / 256)] (``adamw_state`` makes either;
    exp_avg_sqs then hold the root of the second moment).  ``copies``: bfloat16
    tensors that receive the new parameters; ``grad_scale``: a float32 CUDA
    scalar that every gradient is multiplied with."""
    avg_scales, sq_scales = (None, None) if scales is None else scales
    _done(_native.adamw(params, grads, exp_avgs, exp_avg_sqs, avg_scales, sq_scales, copies, grad_scale, lr, betas[0],
                        betas[1], eps, weight_decay, step, _handle(stream)), "zipccl_adamw_step")
