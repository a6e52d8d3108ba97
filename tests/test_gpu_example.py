"""The example that trains a block against a teacher runs, and learns."""
import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "distill_block.py")


def test_distill_block_learns():
    spec = importlib.util.spec_from_file_location("distill_block", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train()
    assert all(math.isfinite(v) and v >= 0 for v in losses)  # a divergence
    assert sum(losses[-5:]) < 0.7 * sum(losses[:5])
    assert losses == example.train()  # seeds decide everything
