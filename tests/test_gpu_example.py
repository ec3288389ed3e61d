"""The example that runs the 8-bit and expert operators together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_and_serve.py")
    spec = importlib.util.spec_from_file_location("train_and_serve", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.fixture(scope="module")
def trained(example):
    return example.train(30, 2048)


def test_training_converges(trained):
    # Each element of an operand is off by at most 2^-4 of itself (half a step of three
    # mantissa bits), so y by about 2^-4 sqrt(2) of its size at most: a mean square
    # per output below 2^-7, half of which is the loss.
    _, losses = trained
    assert losses[-1] < 2.0 ** -8 < 0.02 * losses[0]


@pytest.mark.parametrize("tokens", [1, 16, 64])
def test_serving_agrees_with_float32(example, trained, tokens):
    # Outputs are rounded to bf16 (2^-9 of each element at most); the float32 side's own
    # rounding, and h's 16 bits, are far below the other half of the bar.
    for fmt in example.FORMATS:
        assert max(example.serve(trained[0], tokens, fmt)) < 2.0 ** -8, fmt
