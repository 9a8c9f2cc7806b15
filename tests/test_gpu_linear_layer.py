"""The example layer: a training step, and the same tokens served by prefill and steps."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_served_tokens_match_the_packed_forward():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "linear_layer.py")
    spec = importlib.util.spec_from_file_location("linear_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    # both outputs carry bf16 roundings: of the projections (which differ by their matrix
    # product's order), of the attention's terms and of the result, each 2^-8 at most
    assert mod.main() < 4 * 2.0 ** -8
