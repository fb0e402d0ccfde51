"""CPU check of the training example's torch function: what it refuses."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Reached(Exception):
    """The backward has come to what the forward kept."""


class Kept:
    @property
    def saved_tensors(self):
        raise Reached()


@pytest.fixture(scope="module")
def layer():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        from train_layer import ExpertLayer
    finally:
        sys.path.pop(0)
    return ExpertLayer


def test_a_backward_that_is_to_be_differentiated_is_refused(layer):
    """autograd runs a backward with gradients enabled where create_graph is given."""
    dout = torch.zeros((2, 128), dtype=torch.bfloat16)
    with torch.enable_grad(), pytest.raises(RuntimeError, match="second derivative"):
        layer.backward(Kept(), dout)
    with torch.no_grad(), pytest.raises(Reached):
        layer.backward(Kept(), dout)


def test_create_graph_reaches_the_function_as_enabled_gradients():
    seen = []

    class Same(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return x.clone()

        @staticmethod
        def backward(ctx, d):
            seen.append(torch.is_grad_enabled())
            return d

    x = torch.ones(3, requires_grad=True)
    for create in (False, True):
        torch.autograd.grad(Same.apply(x).sum(), x, create_graph=create)
    assert seen == [False, True]
