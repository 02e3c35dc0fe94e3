"""The attention layer example end to end: its training lowers the loss, and rows decoded from the paged
cache are those of one pass over the whole sequence."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_trains_and_serves():
    import attention_layer as example

    layer, losses = example.train(steps=20)
    assert losses[-1] < 0.7 * losses[0]
    assert all(b < a for a, b in zip(losses[:5], losses[1:6]))
    diff, size = example.serve(layer)
    # bfloat16 rows: half a step for the roundings of P, of the layer's inner result and of its output, on both sides
    assert diff <= 2 * 3 * 2.0 ** -8 * size
