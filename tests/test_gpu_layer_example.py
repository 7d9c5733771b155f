"""The example's int8 layer and its training step of the router and the norm run."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens", [1, 64, 256])
def test_int8_layer(tokens):
    """Differences: bf16's half step of the down product's rows and of the result, 2^-8 each; a value next to a tie that
    goes to the other code, a step of 1 / 127 of its row's largest for few of them."""
    assert _example().serve_int8(tokens=tokens) < 0.02


def test_router_and_norm_gradients():
    """binary32 sums of up to 512 terms; dh is rounded to bf16: half a step, 2^-8."""
    dlogits, dh, dscale = _example().train_router()
    assert dlogits < 1e-4 and dh < 2.0 ** -8 and dscale < 1e-4
