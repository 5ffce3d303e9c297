"""examples/gated_block.py runs the gated feed-forward block's operators together, beside the FP8 down-projection, the
INT8 linear layer and a library product (GPU).

Tensors are bfloat16: a rounding is at most 2^-9 of a value on either side, its rms relative to a tensor's norm at most 2^-9 too.
Forward: one rounding for x, two for h (x's passes both projections, which doubles it in the product: three in all),
one for z, two for y.  FP8 codes (E4M3, 3 bits) round by up to 2^-4, rms below 0.6 of that for each operand: 5.4% together,
and a delayed scale that leaves some codes subnormal; below 7%.  Gradients go through at most six rounded tensors each
(dout, dh, dg or du with the saved gate and up, dx, the residual's sum): 6 x 2^-9, and h's three for the weights of the
down-projection; all below 2^-6.  INT8: 0.85% for the weight's codes and 2.5% for h's (amax up to 13 rms), and h's own
roundings: below 4%.  With the adapters' products: h's roundings and the sum's own, below 2^-7."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_block.py")


def _example():
    spec = importlib.util.spec_from_file_location("gated_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("sizes", [{}, {"tokens": 333, "width": 256, "hidden": 640}])
def test_training_block(sizes):
    errors = _example().training(**sizes)
    limits = {"x": 2.0 ** -9, "h": 3 * 2.0 ** -9, "FP8 down-projection": 0.07, "z": 2.0 ** -9, "y": 2 * 2.0 ** -9}
    assert all(e < limits.get(k, 2.0 ** -6) for k, e in errors.items()), errors


@pytest.mark.parametrize("sizes", [{}, {"tokens": 1}, {"tokens": 300, "width": 333, "hidden": 1001, "rank": 9}])
def test_serving_block(sizes):
    errors = _example().serving(**sizes)
    limits = {"h": 2.0 ** -8, "INT8 down-projection": 0.04, "with adapters": 2.0 ** -7}
    assert all(e < limits[k] for k, e in errors.items()), errors
