"""What the experts compute, from the definitions, in 64 bits and on the host:
8-bit blocks, their products with gradients, the layer for a few tokens."""
from __future__ import annotations

import math

import numpy as np

import operator_reference as ref

BLOCK = 128


def exponents(top):
    """The smallest whole number e from -127 on with top <= 448 * 2^e."""
    out = np.full(np.shape(top), -127, np.int64)
    for i, t in np.ndenumerate(top):
        if t > 0:
            e = max(-127, math.frexp(t)[1] - 10)
            while t > 448 * 2.0 ** e:
                e += 1
            while e > -127 and t <= 448 * 2.0 ** (e - 1):
                e -= 1
            out[i] = e
    return out


def e4m3(y):
    """The nearest value of 4 exponent and 3 mantissa bits, ties to even; NaN for what is not finite."""
    with np.errstate(invalid="ignore"):
        unit = np.exp2(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
        return np.where(np.isfinite(y), np.round(y / unit) * unit, np.nan)


def _top(x, axis):
    return np.where(np.isfinite(x), np.abs(x), 0.0).max(axis=axis, initial=0.0)


def quantize_rows(x):
    """(values of the codes, exponents of the scales)."""
    codes, scales = np.empty_like(x), []
    for k in range(0, x.shape[1], BLOCK):
        e = exponents(_top(x[:, k:k + BLOCK], 1))
        codes[:, k:k + BLOCK] = e4m3(x[:, k:k + BLOCK] * np.exp2(-e.astype(float))[:, None])
        scales.append(e)
    return codes, np.stack(scales, 1) if scales else np.zeros((x.shape[0], 0), np.int64)


def chunks(offsets, rows):
    """Chunks as the kernels take offsets: from 0 on, never falling, within the rows."""
    if offsets is None:
        return [(0, rows)]
    at, out = 0, []
    for o in list(offsets)[1:]:
        upto = max(at, min(max(int(o), 0), rows))
        out.append((at, upto))
        at = upto
    return out


def quantize_columns(x, offsets=None):
    spans = chunks(offsets, x.shape[0])
    codes = np.zeros_like(x)
    scales = np.full((x.shape[0] // BLOCK + len(spans), x.shape[1]), -127, np.int64)
    n = 0
    for a, b in spans:
        for m in range(a, b, BLOCK):
            part = x[m:min(b, m + BLOCK)]
            scales[n] = exponents(_top(part, 0))
            codes[m:min(b, m + BLOCK)] = e4m3(part * np.exp2(-scales[n].astype(float)))
            n += 1
    return codes, scales


def quantize_weights(w):
    codes = np.empty_like(w)
    E, N, K = w.shape
    scales = np.empty((E, -(-N // BLOCK), -(-K // BLOCK)), np.int64)
    for e, i, j in np.ndindex(scales.shape):
        at = np.s_[e, i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
        scales[e, i, j] = exponents(_top(w[at], (0, 1)))
        codes[at] = e4m3(w[at] * 2.0 ** -float(scales[e, i, j]))
    return codes, scales


def rows_values(codes, scales):
    return codes * np.exp2(scales.astype(float)).repeat(BLOCK, 1)[:, :codes.shape[1]]


def weights_values(codes, scales):
    s = np.exp2(scales.astype(float)).repeat(BLOCK, 1)[:, :codes.shape[1]]
    return codes * s.repeat(BLOCK, 2)[:, :, :codes.shape[2]]


def columns_values(codes, scales, offsets=None):
    out = np.zeros_like(codes)
    n = 0
    for a, b in chunks(offsets, codes.shape[0]):
        for m in range(a, b, BLOCK):
            out[m:min(b, m + BLOCK)] = codes[m:min(b, m + BLOCK)] * np.exp2(scales[n].astype(float))
            n += 1
    return out


def matmul(x, w, offsets=None):
    """(rows times their expert's matrix, the same of magnitudes)."""
    y, size = np.zeros((x.shape[0], w.shape[1])), np.zeros((x.shape[0], w.shape[1]))
    for e, (a, b) in enumerate(chunks(offsets, x.shape[0])):
        y[a:b], size[a:b] = x[a:b] @ w[e].T, np.abs(x[a:b]) @ np.abs(w[e]).T
    return y, size


def matmul_weights(g, x, offsets=None):
    spans = chunks(offsets, x.shape[0])
    return (np.stack([g[a:b].T @ x[a:b] for a, b in spans]), np.stack([np.abs(g[a:b]).T @ np.abs(x[a:b]) for a, b in spans]))


def activation(name, v):
    if name == "silu":
        with np.errstate(over="ignore"):
            return v / (1 + np.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + np.vectorize(math.erf)(v / math.sqrt(2)))
    return np.maximum(v, 0)


def layer(x, router, up, down, k, act="silu", residual=None, mask=None, score="softmax", bias=None, groups=1, kept=1,
          group_score="max", renormalize=True, scale=1.0):
    """y, weights, ids, the smallest gap that decided a choice, and the sums of
    magnitudes that y's errors go by."""
    logits = x @ router.T
    w, ids, gap = ref.route(logits, k, score, bias, groups, kept, group_score, renormalize, scale, mask)
    for t in range(len(x)):                     # by the logits themselves there is no gap in the reference
        if mask is None or mask[t]:
            l = np.sort(logits[t])[::-1]
            if len(l) > 1:
                gap = min(gap, float(np.min(l[:min(k, len(l) - 1)] - l[1:min(k, len(l) - 1) + 1])))
    y = np.zeros_like(x) if residual is None else np.array(residual, np.float64)
    size = np.abs(y)
    inner = down.shape[2]
    for t in range(len(x)):
        for j, e in enumerate(ids[t]):
            if e < 0:
                continue
            g, ga = up[e] @ x[t], np.abs(up[e]) @ np.abs(x[t])
            h = activation(act, g[:inner]) * (g[inner:] if up.shape[1] > inner else 1.0)
            ha = ga[:inner] * (ga[inner:] if up.shape[1] > inner else 1.0)
            y[t] += w[t, j] * (down[e] @ h)
            size[t] += np.abs(w[t, j]) * (np.abs(down[e]) @ ha) * (1 + 2 * (np.abs(router) @ np.abs(x[t])).max())
    return y, w, ids, gap, size
