"""The operators around the exchange from their definitions, in 64 bits and on
the host (numpy, one token or pair at a time)."""
from __future__ import annotations

import math

import numpy as np

F32_MAX = float(np.finfo(np.float32).max)
BLOCK = 256


def scores(row, score):
    """float64 scores of one token and which experts are eligible."""
    row = np.minimum(np.asarray(row, np.float64), F32_MAX)
    fit = row > -np.inf
    s = np.zeros(row.size)
    if fit.any():
        if score == "softmax":
            e = np.exp(row[fit] - row[fit].max())
            s[fit] = e / e.sum()
        else:
            with np.errstate(over="ignore"):
                s[fit] = 1.0 / (1.0 + np.exp(-row[fit]))
    return s, fit, row


def choose(row, k, score, bias, groups, kept, group_score):
    """Chosen experts of one token, best first (fewer than k where fewer are
    eligible), and the smallest gap that decided anything."""
    s, fit, l = scores(row, score)
    E = row.size
    by_logit = score == "softmax" and bias is None and (groups == 1 or group_score == "max")
    c = l.copy() if by_logit else s + (0.0 if bias is None else np.asarray(bias, np.float64))
    c[~fit | ~(c > -np.inf)] = -np.inf
    gaps = []
    if groups > 1:
        size = E // groups
        value = []
        for g in range(groups):
            part = np.sort(c[g * size:(g + 1) * size])[::-1]
            part = part[part > -np.inf][:2 if group_score == "top2" else 1]
            value.append(part.sum() if part.size else -np.inf)
        order = sorted(range(groups), key=lambda g: (-value[g], g))
        if kept < groups and value[order[kept]] > -np.inf:
            gaps.append(value[order[kept - 1]] - value[order[kept]])
        for g in order[kept:]:
            c[g * size:(g + 1) * size] = -np.inf
    order = sorted((e for e in range(E) if c[e] > -np.inf), key=lambda e: (-c[e], e))
    gaps += [c[a] - c[b] for a, b in zip(order[:k], order[1:k + 1])]
    gaps = [g for g in gaps if g != 0]
    return order[:k], (min(gaps) if gaps and not by_logit else math.inf)


def weigh(row, ids, score, renormalize, scale):
    s, _, _ = scores(row, score)
    w = s[list(ids)]
    if renormalize:
        if score == "softmax" and len(ids):
            l = np.minimum(np.asarray(row, np.float64)[list(ids)], F32_MAX)
            w = np.exp(l - l.max())
        total = w.sum()
        w = w / total if total > 0 else np.zeros_like(w)
    return w * scale


def route(logits, k, score="softmax", bias=None, groups=1, kept=1, group_score="max", renormalize=True, scale=1.0,
          mask=None):
    T = len(logits)
    ids = np.full((T, k), -1, np.int64)
    w = np.zeros((T, k))
    gap = math.inf
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        got, g = choose(logits[t], k, score, bias, groups, kept, group_score)
        gap = min(gap, g)
        ids[t, :len(got)] = got
        w[t, :len(got)] = weigh(logits[t], got, score, renormalize, scale)
    return w, ids, gap


def route_grad(grad, logits, ids, score, renormalize, scale):
    """By the Jacobians: weights by scores, scores by logits."""
    out = np.zeros(logits.shape)
    for t in range(len(logits)):
        live = [(k, e) for k, e in enumerate(ids[t]) if e >= 0]
        if not live:
            continue
        s, fit, _ = scores(logits[t], score)
        g = np.zeros(s.size)
        for k, e in live:
            g[e] = grad[t, k] * scale
        if renormalize:
            at = [e for _, e in live]
            total = s[at].sum()
            if total == 0:
                continue
            mean = (g[at] * s[at]).sum() / total
            for e in at:
                g[e] = (g[e] - mean) / total
        out[t] = s * (g - (g * s).sum()) if score == "softmax" else g * s * (1 - s)
        out[t][~fit] = 0
    return out


def plan(ids, experts):
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    counts = [int((key == e).sum()) for e in range(experts)]
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    place = list(offsets)
    slots = np.zeros(flat.size, np.int64)
    for i, e in enumerate(key):
        slots[i] = place[e] if e < experts else -1 - place[e]
        place[e] += 1
    return np.array(counts), offsets, slots.reshape(ids.shape)


def dispatch(x, slots):
    rows = np.zeros((slots.size, x.shape[1]))
    for t, line in enumerate(slots):
        for s in line:
            if s >= 0:
                rows[s] = x[t]
    return rows


def combine(rows, slots, weights=None, residual=None):
    y = np.zeros((slots.shape[0], rows.shape[1])) if residual is None else np.array(residual, np.float64)
    size = np.abs(y)
    for t, line in enumerate(slots):
        for k, s in enumerate(line):
            if s >= 0:
                add = (1.0 if weights is None else float(weights[t, k])) * rows[s]
                y[t] += add
                size[t] += np.abs(add)
    return y, size


def combine_grad(grad, rows, slots, weights=None):
    gr = np.zeros(rows.shape)
    gw = np.zeros(slots.shape)
    size = np.zeros(slots.shape)
    for t, line in enumerate(slots):
        for k, s in enumerate(line):
            if s >= 0:
                gr[s] = (1.0 if weights is None else float(weights[t, k])) * grad[t]
                gw[t, k] = (grad[t] * rows[s]).sum()
                size[t, k] = np.abs(grad[t] * rows[s]).sum()
    return gr, gw, size


def adamw(p, g, m, v, step, lr, betas, eps, weight_decay, grad_scale=1.0):
    b1, b2 = betas
    g = g * grad_scale
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    with np.errstate(divide="ignore", invalid="ignore"):
        change = lr / (1 - b1 ** step) * m / (np.sqrt(v / (1 - b2 ** step)) + eps)
    return p * (1 - lr * weight_decay) - change, m, v, change


def e4m3_step(y):
    """Distance between neighbouring E4M3 values at |y|."""
    y = np.maximum(np.abs(y), 2.0 ** -6)
    return np.exp2(np.floor(np.log2(y)) - 3)
