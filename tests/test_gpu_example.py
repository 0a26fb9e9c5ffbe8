"""The example of a 4-bit mixture-of-experts layer runs, on both sides of the tensor-core path."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tokens", [1, 48, 200])
def test_moe_layer_example(lib, tokens):
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    errors = m.main(tokens)
    # bf16 outputs: half an ulp is at most 2^-9 of each value
    assert errors["projection"] < 2.0 ** -9 and errors["experts"] < 2.0 ** -8
    assert errors["gradient of a constant"] < 1e-5
