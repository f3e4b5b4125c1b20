"""CPU checks of the training example's autograd wrappers, with torch in place of the
library's calls: gradients reach the right arguments, and a second derivative raises
instead of losing the operators' part of it."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytest.importorskip("clebsch_gordan_tensor_node_amd")
import train_potential as E  # noqa: E402


class _Calls:
    """Stands for the package: y = x w + b and the like, in torch."""

    @staticmethod
    def layer_norm_forward(x, w, b):
        return x * x * w + b, torch.zeros(2, x.shape[0])

    @staticmethod
    def layer_norm_backward(g, x, stats, w):
        return 2 * g * x * w, (g * x * x).sum(0), g.sum(0)

    @staticmethod
    def irreps_norm_forward(plan, x, w, b):
        return _Calls.layer_norm_forward(x, w, b)

    @staticmethod
    def irreps_norm_backward(plan, g, x, stats, w):
        return _Calls.layer_norm_backward(g, x, stats, w)

    @staticmethod
    def conv_forward(plan, pos, x, w):
        return x * x * w

    @staticmethod
    def conv_backward(plan, pos, x, w, g, need):
        return 2 * g * x * w, (g * x * x).sum(0), None


def _wrapped(name):
    gen = torch.Generator().manual_seed(0)
    x, w, b = (torch.randn(*s, generator=gen, dtype=torch.float64).requires_grad_() for s in ((5, 3), (3,), (3,)))
    if name == "LayerNorm":
        return (x, w, b), lambda: E.LayerNorm.apply(x, w, b)
    if name == "IrrepsNorm":
        return (x, w, b), lambda: E.IrrepsNorm.apply(None, x, w, b)
    return (x, w), lambda: E.Conv.apply(None, (None,), x, w)


@pytest.mark.parametrize("name", ["LayerNorm", "IrrepsNorm", "Conv"])
def test_wrappers_differentiate_once(name, monkeypatch):
    monkeypatch.setattr(E, "C", _Calls)
    inputs, call = _wrapped(name)
    got = torch.autograd.grad(call().square().sum(), inputs)
    x, w, b = inputs if len(inputs) == 3 else (*inputs, 0.0)
    want = torch.autograd.grad((x * x * w + b).square().sum(), inputs)
    assert all(torch.allclose(a, c) for a, c in zip(got, want))
    x, w = inputs[:2]
    first = torch.autograd.grad(call().square().sum(), inputs, create_graph=True)
    for second in (lambda: torch.autograd.grad(sum(g.sum() for g in first), inputs),
                   lambda: torch.autograd.grad(first[0].square().sum() + x.square().sum() + w.sum(), (x, w)),
                   lambda: (first[1].sum() + w.sum()).backward()):
        with pytest.raises(RuntimeError, match="second derivative"):
            second()
