"""examples/mlp_block.py runs the operators around the MLP together (GPU).

Training tensors are bfloat16: one rounding (2^-9 of a value, rms a third of half a step, below 2^-9) each
for z and dz, two in a row for y (z's rounding passes the norm) and for nothing else; sums over 2048
tokens of unrounded products see z's rounding only.  All stay below 2^-8 relative to the norm.
Serving: INT8 codes of a normal row are off by a uniform error of one step / 12^0.5, a step being
amax / 127, amax about 3.3 (width 768) to 3.7 (2048) standard deviations: 0.75% to 0.85% per operand;
up-projection 1.2% with both operands' errors, the squared ReLU doubles that (2.4%), its own cast is of a
heavier tail (amax about 13 of rms 1.2: 2.5%), the down-projection's weights 0.85%: 3.6% together, below 6%."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mlp_block.py")


def _example():
    spec = importlib.util.spec_from_file_location("mlp_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_training_tail():
    errors = _example().training(tokens=999, width=1001)
    assert all(e < 2.0 ** -8 for e in errors.values()), errors
    errors = _example().training()
    assert all(e < 2.0 ** -8 for e in errors.values()), errors


def test_serving_block():
    for sizes in ({}, {"prompt": 77, "width": 500, "hidden": 1001}):
        errors = _example().serving(**sizes)
        assert all(e < 0.06 for e in errors.values()), errors
