"""examples/hybrid_layer.py: the recurrence and the attention-layer operators together.

Tolerances: outputs are sums of bf16 products whose operands are rounded at each of about six
steps (2^-8 each, of values the size of the largest): 6 * 2^-8 = 2.4e-2 between decode and prefill,
which round at different places.  The gradient is compared along itself with a difference over
steps of 2% of x: second-order terms cancel, rounding of the inputs' steps is 2^-8 / 0.02 of a step's
entries but random over 200 000 of them; 5%."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_serving_and_training(gdn):
    import hybrid_layer

    model = hybrid_layer.Hybrid()
    assert hybrid_layer.serve_check(model) <= 2.4e-2
    grad, diff = hybrid_layer.train_check(model)
    assert abs(grad - diff) <= 0.05 * abs(grad)
