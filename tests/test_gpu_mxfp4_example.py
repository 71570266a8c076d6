"""The 4-bit operators together, as the example runs them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tokens", [1, 5, 24])
def test_decoder_step(mhr, tokens):
    spec = importlib.util.spec_from_file_location(
        "mxfp4_decoder_step", os.path.join(ROOT, "examples", "mxfp4_decoder_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # both blocks round to bf16 four times (2^-8 each at most, of values no larger than a few
    # times the result's)
    assert example.main(tokens=tokens, steps=2) < 4 * 2.0 ** -8
