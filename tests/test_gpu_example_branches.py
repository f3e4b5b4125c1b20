"""The training example with routed edges on the GPU: it runs, repeats bit for bit, and its
gradients match differences of the loss."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytest.importorskip("clebsch_gordan_tensor_node_amd")
import train_potential as E  # noqa: E402
import workloads as WL  # noqa: E402

pytestmark = pytest.mark.gpu


def test_example_runs_with_branches():
    losses = E.train("tiny", steps=12, bits=32, branches=3)
    assert len(losses) == 12 and all(v == v and v < 1e6 for v in losses)
    assert losses == E.train("tiny", steps=12, bits=32, branches=3)


@pytest.mark.parametrize("branches", [1, 2])
def test_example_gradients_with_branches(branches):
    # every branch is chosen, so that the loss is smooth; the slope of the balance loss, whose
    # counts are held fixed, is 1 for each branch then
    net = E.Potential(WL.WORKLOADS["tiny"], torch.device("cuda:0"), branches=branches)
    target = torch.randn(net.pos.shape[0], generator=torch.Generator().manual_seed(1)).cuda()

    def loss():
        energies, balance = net.energies_and_balance()
        return (energies - target).square().mean() + 0.5 * balance

    grads = torch.autograd.grad(loss(), net.values)
    gen = torch.Generator().manual_seed(2)
    for name, v, g in zip(net.names, net.values, grads):
        d = torch.randn(v.shape, generator=gen).cuda()
        d /= d.norm()
        h = 1e-2
        with torch.no_grad():
            v += h * d
            up = loss().double()
            v -= 2 * h * d
            down = loss().double()
            v += h * d
        diff, want = float((up - down) / (2 * h)), float((g * d).sum())
        # as without branches: fp32 losses of order 2 differ by some 1e-6 / 2h = 1e-4; the third
        # derivative times h^2/6 is below a hundredth of the gradient's scale
        assert abs(diff - want) < 2e-3 + 2e-2 * abs(want), (name, diff, want)


def test_example_has_no_second_derivative_through_branches():
    net = E.Potential(WL.WORKLOADS["tiny"], torch.device("cuda:0"), branches=2)
    grads = torch.autograd.grad(net.energies().square().sum(), net.values, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        sum(g.square().sum() for g in grads).backward()


def test_example_gradients_with_more_branches_than_chosen(monkeypatch):
    # two of three branches: the choices have to stay as they are within the step, or the loss jumps
    # (the second and third logits of an edge are 0.04 apart at the least)
    net = E.Potential(WL.WORKLOADS["tiny"], torch.device("cuda:0"), branches=3)
    target = torch.randn(net.pos.shape[0], generator=torch.Generator().manual_seed(1)).cuda()
    routes, forward = [], E.C.route_forward
    monkeypatch.setattr(E.C, "route_forward", lambda *a, **k: routes.append(forward(*a, **k)) or routes[-1])

    def loss():
        energies, balance = net.energies_and_balance()
        return (energies - target).square().mean() + 0.5 * balance

    grads = torch.autograd.grad(loss(), net.values)
    assert all((g != 0).any() for g in grads)
    first = routes[0].ids.clone()
    assert (first >= 0).all() and routes[0].counts.sum() == 2 * len(first) and (routes[0].counts > 0).all()
    gen = torch.Generator().manual_seed(2)
    for name, v, g in zip(net.names, net.values, grads):
        d = torch.randn(v.shape, generator=gen).cuda()
        d /= d.norm()
        h = 1e-3
        with torch.no_grad():
            v += h * d
            up = loss().double()
            v -= 2 * h * d
            down = loss().double()
            v += h * d
        assert all(torch.equal(r.ids, first) for r in routes[-2:]), name
        diff, want = float((up - down) / (2 * h)), float((g * d).sum())
        # fp32 losses of order 2 differ by some 1e-6 / 2h = 5e-4; the third derivative times h^2/6 is
        # below a ten thousandth of the gradient's scale
        assert abs(diff - want) < 2e-3 + 2e-2 * abs(want), (name, diff, want)
