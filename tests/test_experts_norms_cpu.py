"""Mistakes planted in the reference: the bound that the GPU's layer is held to lets none of them pass."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import experts_norms as norms  # noqa: E402
from experts_norms import ex, values  # noqa: E402

TYPES = [torch.float32, torch.bfloat16, torch.float16]
CASES = [
    # tokens, hidden, inner, experts, top_k, gated, activation
    (1, 256, 128, 8, 2, True, "silu"), (3, 520, 201, 6, 2, False, "gelu"), (7, 130, 65, 70, 3, True, "gelu"),
    (8, 64, 300, 33, 8, True, "relu"), (9, 257, 64, 12, 4, True, "silu"), (32, 100, 60, 4, 4, True, "silu"), (5, 2050, 129, 9, 3, True, "silu"),
]


def eleven_bits(a):
    """What a single 19-bit operand holds of a float."""
    return np.ldexp(np.round(np.ldexp(np.frexp(a)[0], 11)), np.frexp(a)[1] - 11)


def mistakes(x, router, up, down, k, act, residual, dtype):
    inner = down.shape[2]
    yield "another activation", ex.layer(x, router, up, down, k, {"silu": "gelu", "gelu": "relu", "relu": "silu"}[act], residual)[0]
    shorter = down.copy()
    shorter[:, :, inner - 1] = 0
    yield "the last place left out", ex.layer(x, router, up, shorter, k, act, residual)[0]
    shorter[:, :, inner // 2:] = 0
    yield "half the places left out", ex.layer(x, router, up, shorter, k, act, residual)[0]
    yield "no experts", residual
    y, w, ids, _, _ = ex.layer(x, router, up, down, k, act, residual)
    swapped = np.concatenate([up[:, inner:], up[:, :inner]], 1) if up.shape[1] > inner else up * 1.01
    yield "gate and value exchanged, or a hundredth more", ex.layer(x, router, swapped, down, k, act, residual)[0]
    without = np.array(y)
    for t in range(len(x)):  # each token's last expert
        e = ids[t, -1]
        g = up[e] @ x[t]
        without[t] -= w[t, -1] * (down[e] @ (ex.activation(act, g[:inner]) * (g[inner:] if up.shape[1] > inner else 1.0)))
    yield "an expert left out", without
    if dtype == torch.float32:
        for name, cut in (("x", (eleven_bits(x), router, up, down)), ("up", (x, router, eleven_bits(up), down)), ("down", (x, router, up, eleven_bits(down)))):
            yield "11 bits of " + name, ex.layer(*cut, k, act, residual)[0]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:5])) + f"-{c[6]}")
def test_the_bound_refuses_wrong_layers(case, dtype):
    rng = np.random.default_rng(sum(case[:5]))
    x, router, up, down, residual = map(values, norms.draw(rng, case, dtype))
    k, act = case[4], case[6]
    y, w, _, _, _ = ex.layer(x, router, up, down, k, act, residual)
    assert norms.off(norms.rounded(y, dtype), y, residual, dtype) == 0
    for what, wrong in mistakes(x, router, up, down, k, act, residual, dtype):
        assert norms.off(norms.rounded(wrong, dtype), y, residual, dtype) > 3, what
    if dtype == torch.float32 and k > 1:
        assert norms.weights_off(ex.layer(x, eleven_bits(router), up, down, k, act, residual)[1], w) > 3
