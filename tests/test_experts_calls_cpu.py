"""Arguments of the experts' calls that are neither taken nor refused by their type alone."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
import lossless_bf16_tensor_zipccl_gb300 as zc  # noqa: E402
from test_operators_tensors_cpu import here  # noqa: E402


def test_a_by_rows_that_is_neither_true_nor_false_raises_its_own_error():
    with pytest.raises(RuntimeError, match="Boolean value"):
        zc.moe_quantize_columns(here(4, 256), by_rows=torch.tensor([True, False]))
