"""The router-training example end to end: the operators together on the tiny
layer. The balance loss of even loads and probabilities is 1; the lopsided
router starts above it and the steps bring it down."""
import os
import sys

import pytest

import gpu_helpers as gh

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


def test_example_balances_the_router():
    gh.lib()
    import router_training
    history = router_training.train(steps=25, verbose=False)
    first, last = history[0], history[-1]
    assert first[0] > 1.05
    assert last[0] < 1.0 + 0.5 * (first[0] - 1.0)
    assert last[2] < first[2]
    # the same steps again give the same numbers, bit for bit
    assert router_training.train(steps=3, verbose=False) == history[:3]
