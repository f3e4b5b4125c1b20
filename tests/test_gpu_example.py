"""The training example end to end on the GPU: with 32-bit and with 8-bit moments the
32-atom potential fits its targets, and its gradients match differences of the loss."""
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


@pytest.mark.parametrize("bits", [32, 8])
def test_example_learns(bits):
    losses = E.train("tiny", steps=150, bits=bits)
    print(f"{bits}-bit moments: loss {losses[0]:.4f} -> {losses[-1]:.4f}", flush=True)
    assert all(v == v for v in losses) and losses[-1] < 0.2 * losses[0]


def test_example_repeats_bitwise():
    assert E.train("tiny", steps=10, bits=8) == E.train("tiny", steps=10, bits=8)


def test_example_gradients():
    net = E.Potential(WL.WORKLOADS["tiny"], torch.device("cuda:0"))
    target = torch.randn(net.pos.shape[0], generator=torch.Generator().manual_seed(1)).cuda()

    def loss():
        return (net.energies() - target).square().mean()

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
        # fp32 losses of order 2 differ by some 1e-6 / 2h = 1e-4; the third derivative times h^2/6
        # is below a hundredth of the gradient's scale
        assert abs(diff - want) < 2e-3 + 2e-2 * abs(want), (name, diff, want)
