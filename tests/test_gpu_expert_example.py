"""The example of an expert layer: it learns, and its 4-bit weights serve."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_expert_layer_example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import expert_layer
    losses, worst = expert_layer.main(verbose=False)
    assert losses[-1] < 0.5 * losses[0]
    # Rounding a weight to 15 steps over its group's range (about 5 standard deviations)
    # is off by a tenth of a deviation: two layers of that stay well under a third.
    assert worst < 1 / 3
