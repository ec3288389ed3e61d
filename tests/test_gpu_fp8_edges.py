"""The 8-bit operators where nothing, or nothing finite, comes in."""
import numpy as np
import pytest
import torch

import fp8_ref as ref
import microscaling_fp4_quantization_amd as fq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROW, TILE = fq.B128_ROW, fq.B128_TILE


@pytest.mark.parametrize("shape", [(2, 3, 0), (0, 3, 0), (3, 0), (0,), (2, 0, 16), (0, 2, 16)])
def test_linear_of_empty_inputs(shape):
    """Any number of dimensions, no features or no tokens: zeros of the right shapes."""
    x = torch.zeros(shape, device=DEV, requires_grad=True)
    w = torch.zeros(5, shape[-1], device=DEV, requires_grad=True)
    y = fq.fp8_linear(x, w)
    assert y.shape == (*shape[:-1], 5) and not y.any()
    y.backward(torch.ones_like(y))
    assert x.grad.shape == shape and w.grad.shape == w.shape and not x.grad.any() and not w.grad.any()
    assert fq.fp8_linear(x, w[:0]).shape == (*shape[:-1], 0)
