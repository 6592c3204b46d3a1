"""How far a layer's answer is from the one in 64 bits, in units of what its arithmetic
allows: by the norm of what the experts add, not by the magnitudes of all terms.

The unit.  Operands take part with 2^-22 of themselves at most, h with 2^-21, each
instruction cuts 2^-23 of its sum, four and up to twelve of them in a chain.  A sum of
n terms of either sign grows as its errors do, with the root of n: in the norm a
product's error is 2^-21 of it, both factors of h 2^-20, and with the second product
and the weights (2^-20) 2^-19 in all.  2^-18 leaves that twice.  An operand that has
lost its second part is off by 2^-12, an activation, a place or an expert by more.
Results are rounded once beside that: half a step of each value.

Weights: a logit of a size l is off by 2^-21 l in the norm, a weight by the
difference of two of them: 2^-17 of itself for logits up to 8."""
from __future__ import annotations

import numpy as np
import torch

import experts_reference as ex

LAYER, WEIGHTS = 2.0 ** -18, 2.0 ** -17


def draw(rng, case, dtype, router_dtype=None):
    """x, router, up, down and residual on the host; the nearest logits that decide are 1e-4 apart."""
    tokens, hidden, inner, experts, k, gated, _ = case
    up = torch.from_numpy(rng.normal(size=(experts, inner * (2 if gated else 1), hidden)) * hidden ** -0.5).to(dtype)
    down = torch.from_numpy(rng.normal(size=(experts, hidden, inner)) * inner ** -0.5).to(dtype)
    residual = torch.from_numpy(rng.normal(size=(tokens, hidden))).to(dtype)
    router = torch.from_numpy(rng.normal(size=(experts, hidden)) * 2 * hidden ** -0.5).to(router_dtype or dtype)
    x = torch.from_numpy(rng.normal(size=(tokens, hidden))).to(dtype)
    for _ in range(200):
        l = np.sort(values(x) @ values(router).T, 1)[:, ::-1][:, :k + 1]
        bad = (l[:, :-1] - l[:, 1:] < 1e-4).any(1)
        if not bad.any():
            return x, router, up, down, residual
        x[bad] = torch.from_numpy(rng.normal(size=(int(bad.sum()), hidden))).to(dtype)
    raise AssertionError("no settled draw")


def values(t):
    return t.double().cpu().numpy()


def off(got, want, residual, dtype):
    """The norm of what rounding once does not explain, in units of the norm of what the experts add."""
    once = 1.001 * torch.finfo(dtype).eps / 2 * np.abs(want)
    if dtype == torch.float16:
        once = np.maximum(once, 2.0 ** -25)
    part = np.linalg.norm(want if residual is None else want - residual)
    left = np.linalg.norm(np.maximum(np.abs(got - want) - once, 0))
    return left / (LAYER * part) if part else left


def weights_off(got, want):
    """Largest relative error of a weight, in units."""
    return float((np.abs(got - want) / (WEIGHTS * np.maximum(np.abs(want), 1e-30))).max())


def rounded(y, dtype):
    return values(torch.from_numpy(y).to(dtype))


__all__ = ["LAYER", "WEIGHTS", "draw", "ex", "off", "rounded", "values", "weights_off"]
