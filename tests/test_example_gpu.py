"""The operators and the compressed exchanges together: a few training steps of
the example learn, and learn alike with states in 8 and in 32 bits."""
from __future__ import annotations

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("moe_training_step", os.path.join(ROOT, "examples", "moe_training_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_training_steps_learn(example):
    runs = {bits: example.train(steps=25, ranks=2, tokens=700, hidden=200, experts=6, bits=bits) for bits in (8, 32)}
    for losses, ratio in runs.values():
        assert losses[-1] < 0.7 * losses[0]
        assert 0.6 < ratio < 0.8          # 10.6 bits of 16 for Gaussian values, headers of small chunks
    assert abs(runs[8][0][-1] - runs[32][0][-1]) < 0.1 * runs[32][0][-1]
