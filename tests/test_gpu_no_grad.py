"""Linear layers under torch.no_grad() and inference_mode: the forward pass alone, without what a
backward pass would need, and the same values."""
import sys

import pytest
import torch

import microscaling_fp4_quantization_amd as fq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Calls:
    """The library, with the arguments of its calls kept by name."""

    def __init__(self, lib):
        self._lib, self.seen = lib, []

    def __getattr__(self, name):
        f = getattr(self._lib, name)

        def call(*args):
            self.seen.append((name, args))
            return f(*args)

        return call


@pytest.fixture
def calls(monkeypatch):
    kept = Calls(fq.lib())
    for module in ("grouped", "fp8_linear"):  # (fq.fp8_linear is the function)
        monkeypatch.setattr(sys.modules[f"{fq.__name__}.{module}"], "lib", lambda: kept)
    return kept


def forward_flags(calls, name, at):
    """(want_dx, want_dw, saved, its bytes) of each forward call."""
    return [tuple(a[at:at + 4]) for n, a in calls.seen if n == name]


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
@pytest.mark.parametrize("x_grad", [False, True])
def test_grouped_linear(calls, mode, x_grad):
    x = torch.randn(300, 256, device=DEV, requires_grad=x_grad)
    w = torch.nn.Parameter(torch.randn(4, 128, 256, device=DEV))
    offsets = torch.tensor([0, 100, 100, 250, 300], dtype=torch.int32, device=DEV)
    want = fq.fp8_grouped_linear(x, w, offsets)
    with mode():
        y = fq.fp8_grouped_linear(x, w, offsets)
        assert not y.requires_grad and torch.equal(y, want)
    trained, alone = forward_flags(calls, "fp8_grouped_linear_forward", 10)
    assert trained[0] == x_grad and trained[1] and trained[3] > 0
    assert not alone[0] and not alone[1] and alone[2:] == (None, 0)
    want.sum().backward()  # the call in between took nothing from it
    assert w.grad is not None and bool(w.grad[0].any()) and not bool(w.grad[1].any())


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_linear(calls, mode):
    x = torch.randn(3, 70, 256, device=DEV, requires_grad=True)
    w = torch.nn.Parameter(torch.randn(128, 256, device=DEV))
    want = fq.fp8_linear(x, w)
    with mode():
        y = fq.fp8_linear(x, w)
        assert not y.requires_grad and torch.equal(y, want)
    trained, alone = forward_flags(calls, "fp8_linear_forward", 8)
    assert trained[0] and trained[1] and trained[3] > 0
    assert not alone[0] and not alone[1] and alone[2:] == (None, 0)


def test_checkpointed_layers():
    """A forward pass without gradients, done again with them in the backward pass: the same gradients."""
    from torch.utils.checkpoint import checkpoint
    offsets = torch.tensor([0, 90, 200], dtype=torch.int32, device=DEV)
    x = torch.randn(200, 64, device=DEV, requires_grad=True)
    w = torch.randn(2, 96, 64, device=DEV, requires_grad=True)
    v = torch.randn(32, 96, device=DEV, requires_grad=True)
    net = lambda t: fq.fp8_linear(torch.relu(fq.fp8_grouped_linear(t, w, offsets)), v)
    want = torch.autograd.grad(net(x).square().sum(), (x, w, v))
    for reentrant in (False, True):
        x.grad = w.grad = v.grad = None
        checkpoint(net, x, use_reentrant=reentrant).square().sum().backward()
        assert all(torch.equal(a, b) for a, b in zip((x.grad, w.grad, v.grad), want))
