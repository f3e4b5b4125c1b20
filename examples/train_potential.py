"""Trains a one-layer equivariant potential with the library's kernels: the whole path that
a network around the convolution takes, on synthetic energies.

    python examples/train_potential.py [--steps 200] [--bits 8] [--workload tiny]

Every edge's convolution weights come from a radial network (layer norm inside), the
convolution's output is normalised term by term (irreps norm), its scalars give the
energy, and the gradients pass back through the same operators into AdamW, clipped by
their norm on the device.  Dense products and pointwise functions are torch's.  The
operators have first derivatives only: a second one (create_graph=True, forces in the loss)
raises.
"""
import argparse
import math
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import clebsch_gordan_tensor_node_amd as C  # noqa: E402
import workloads as WL  # noqa: E402


class Derivative(torch.autograd.Function):
    """Gradients call(*tensors) that depend on the tensors and cannot be differentiated: a
    second derivative that passes through them raises, and no part of it is lost."""

    @staticmethod
    def forward(ctx, call, *tensors):
        return call(*tensors)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the library's operators have no second derivative")


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        y, stats = C.layer_norm_forward(x, weight, bias)
        ctx.save_for_backward(x, stats, weight)
        return y

    @staticmethod
    def backward(ctx, grad):
        x, stats, weight = ctx.saved_tensors
        return Derivative.apply(lambda g, x, w: C.layer_norm_backward(g, x, stats, w), grad.contiguous(), x, weight)


class IrrepsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, x, weight, bias):
        y, stats = C.irreps_norm_forward(plan, x, weight, bias)
        ctx.plan = plan
        ctx.save_for_backward(x, stats, weight)
        return y

    @staticmethod
    def backward(ctx, grad):
        x, stats, weight = ctx.saved_tensors
        return (None, *Derivative.apply(lambda g, x, w: C.irreps_norm_backward(ctx.plan, g, x, stats, w),
                                        grad.contiguous(), x, weight))


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, graph, x, w):
        ctx.plan, ctx.graph = plan, graph
        ctx.save_for_backward(x, w)
        return C.conv_forward(plan, *graph, x, w)

    @staticmethod
    def backward(ctx, grad):
        x, w = ctx.saved_tensors
        return (None, None, *Derivative.apply(lambda g, x, w: C.conv_backward(ctx.plan, *ctx.graph, x, w, g,
                                                                              need=("x", "w"))[:2], grad.contiguous(), x, w))


class Potential:
    """Parameters and energy of the network on a fixed neighbour list."""

    def __init__(self, wl, device, n_radial=16, hidden=64, seed=0):
        gen = torch.Generator().manual_seed(seed)
        pos, box, cell, _ = WL.positions(wl)
        self.pos = torch.from_numpy(pos).to(device)
        row_ptr, col, shift = C.neighbors_build(self.pos, box, wl.cutoff)
        self.plan = C.Plan(wl.irreps_in, wl.irreps_sh, wl.l_out_max, wl.rule)
        self.norm = C.NormPlan(self.plan.irreps_out)
        self.graph = (self.pos, cell, row_ptr, col, shift)
        # edge lengths in a basis of Gaussians (fixed: the positions do not move here)
        recv = torch.repeat_interleave(torch.arange(len(pos), device=device), (row_ptr[1:] - row_ptr[:-1]).long())
        r = self.pos[col.long()] - self.pos[recv] + shift.float() @ torch.as_tensor(np.asarray(cell, dtype=np.float32).reshape(3, 3), device=device)
        at = torch.linspace(0, wl.cutoff, n_radial, device=device)
        self.basis = torch.exp(-((r.norm(dim=1, keepdim=True) - at) / (wl.cutoff / n_radial)) ** 2)
        f, w = self.plan.f_in, self.plan.w_per_edge

        def normal(*shape, scale=1.0):
            return (scale * torch.randn(*shape, generator=gen)).to(device)

        # name: (value, weight decay); norms and biases are not decayed
        p = {"x": (normal(len(pos), f), 0.0),
             "radial_in": (normal(n_radial, hidden, scale=1 / math.sqrt(n_radial)), 0.01),
             "ln_weight": (torch.ones(hidden, device=device), 0.0), "ln_bias": (torch.zeros(hidden, device=device), 0.0),
             "radial_out": (normal(hidden, w, scale=1 / math.sqrt(hidden)), 0.01),
             "norm_weight": (torch.ones(self.norm.n_weights, device=device), 0.0),
             "norm_bias": (torch.zeros(self.norm.n_biases, device=device), 0.0),
             "readout": (normal(self.norm.n_biases, 1, scale=1 / math.sqrt(self.norm.n_biases)), 0.01)}
        self.names = list(p)
        self.values = [v.requires_grad_() for v, _ in p.values()]
        self.decay = [d for _, d in p.values()]

    def energies(self):
        """One energy per atom [n]: the normalised scalars of the convolution, read out."""
        q = dict(zip(self.names, self.values))
        hidden = LayerNorm.apply(self.basis @ q["radial_in"], q["ln_weight"], q["ln_bias"])
        w = torch.nn.functional.silu(hidden) @ q["radial_out"]
        out = IrrepsNorm.apply(self.norm, Conv.apply(self.plan, self.graph, q["x"], w), q["norm_weight"], q["norm_bias"])
        return (out[:, :self.norm.n_biases] @ q["readout"]).squeeze(1)   # 0e terms lead the output irreps


def train(workload="tiny", steps=200, bits=32, lr=1e-2, device="cuda:0", report=None):
    """The losses of `steps` steps towards random target energies."""
    net = Potential(WL.WORKLOADS[workload], torch.device(device))
    target = torch.randn(net.pos.shape[0], generator=torch.Generator().manual_seed(1)).to(device)
    params = C.ParamSet(net.values, net.decay)
    values = params.pointers([v.detach() for v in net.values])   # the same storage
    state = C.adamw_state(params, bits)
    losses = []
    for t in range(1, steps + 1):
        loss = (net.energies() - target).square().mean()
        grads = params.pointers([g.contiguous() for g in torch.autograd.grad(loss, net.values)])
        factor = C.grad_norm(params, grads, max_norm=1.0)[1:]
        C.adamw_step(params, values, grads, state, lr=lr, step=t, grad_scale=factor, seed=t)
        losses.append(loss.detach())
        if report and t % report == 0:
            print(f"step {t}: loss {losses[-1].item():.4f}", flush=True)
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--bits", type=int, choices=(8, 32), default=32, help="of AdamW's moments")
    ap.add_argument("--workload", default="tiny", choices=("tiny", "c1_768", "c2_768", "si_mask"))
    a = ap.parse_args()
    got = train(a.workload, a.steps, a.bits, report=max(1, a.steps // 10))
    print(f"loss {got[0]:.4f} -> {got[-1]:.4f}")
