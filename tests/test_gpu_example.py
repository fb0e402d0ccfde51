"""The example that trains the router on its balance loss and serves the layer in MXFP4."""
import os
import sys

import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_balances_the_router_and_runs_the_4_bit_layer():
    need_gpu()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import mxfp4_layer
    finally:
        sys.path.pop(0)
    history, off = mxfp4_layer.main(tokens=1000, steps=20)
    (first, counts0), (last, counts1) = history[0], history[-1]
    assert float(last[0]) < float(first[0]) and float(last[0]) >= 0.99
    assert int(counts1.max()) < int(counts0.max())
    assert int(counts0.sum()) == int(counts1.sum()) == (1000 - 125) * 4
    # e2m1 keeps 2 to 3 bits: 0.25 / sqrt(12) .. of a value per operand, four
    # quantised operands on the way; a wrong scale or order would give about 1
    assert 0.02 < off < 0.5
