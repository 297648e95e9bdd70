"""The example that trains an MLP block with the layer operators and LoCo's low-bit path."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_mlp_block_trains(gpu_lib):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import mlp_step
    finally:
        sys.path.pop(0)
    losses = mlp_step.train(tokens=1000, hidden=256, inner=512, steps=40)
    assert all(b == b for b in losses)
    assert losses[-1] < 0.5 * losses[0], losses
