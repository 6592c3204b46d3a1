"""The layer for a few tokens where its answers are known exactly, or to a few
units of 32 bits: what a tolerance by the magnitudes of all terms would let pass.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import lossless_bf16_tensor_zipccl_gb300 as zc  # noqa: E402

TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    zc.load()
    yield
    torch.cuda.synchronize()
    zc.moe_status()          # no wait inside a kernel has run out


@pytest.mark.parametrize("blocks", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("inner", [200, 1100])
def test_layer_holds_21_bits_of_h(inner, dtype, blocks):
    """h = 1 + 2^-9 + m 2^-20, m from 0 to 15, and results that are differences of two of them: (m - n) 2^-20,
    exact in every type.  16 bits of h, in two parts of 8, leave 0."""
    torch.manual_seed(1)
    hidden, tokens = 160, 5
    m = torch.randint(0, 16, (inner,), device="cuda").double()
    up = torch.zeros(1, inner, hidden, dtype=torch.float64, device="cuda")
    up[0, :, 0], up[0, :, 1], up[0, :, 2] = 1, m * 2.0 ** -12, 0.5
    x = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda")
    x[:, 0], x[:, 1], x[:, 2] = 1, 2.0 ** -8, 2.0 ** -8
    down = torch.zeros(1, hidden, inner, dtype=torch.float64, device="cuda")
    row = torch.arange(hidden, device="cuda")
    plus, minus = row % inner, (row * 7 + inner // 2) % inner
    down[0, row, plus] += 1
    down[0, row, minus] -= 1
    matrices = [w.to(dtype) for w in (up, down)]
    if blocks:
        matrices = [zc.moe_quantize_weights(w) for w in matrices]
    y, weights, _ = zc.moe_layer(x.to(dtype), torch.ones(1, hidden, dtype=dtype, device="cuda"), *matrices, 1, activation="relu")
    assert (weights == 1).all()
    assert torch.equal(y.double(), ((m[plus] - m[minus]) * 2.0 ** -20).expand(tokens, hidden))
