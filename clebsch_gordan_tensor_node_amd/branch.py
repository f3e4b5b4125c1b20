"""Operators for a network whose edges go through several branches, each a convolution that
takes its edges' gates: group normalisation with an activation over the rows of each
structure, routing with its balance loss, and the gradient of the convolution's gate.

Argument marshalling over libcgtp.so as in train.py, whose operators these stand beside:
results carry no autograd history, there are no second derivatives, and the formulas stand
in include/cgtp.h beside each entry point.

    hidden, stats = group_norm_forward(rows, 8, gamma, beta, samples=edge_offsets, activation="silu")
    route = route_forward(hidden @ router, k=2, dense=True)
    outs = [conv_forward(plan, *graph, x, w[b], gate=route.gates[b]) for b in range(n)]
    ...
    for b in range(n):
        grad_x, grad_w, _ = conv_backward(plan, *graph, x, w[b], grad_out[b], gate=route.gates[b], need=("x", "w"))
        conv_gate_backward(w[b], grad_w, route.gates[b], out=grad_gates[b])
    grad_logits = route_backward(logits, route, grad_gates, grad_balance)
    grad_rows, grad_gamma, grad_beta = group_norm_backward(grad_hidden, rows, stats, 8, gamma, beta, samples=edge_offsets,
                                                           activation="silu")
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from ._lib import ACT, ELEM, check, load
from .train import _at, _on, _raw_stream, _room, _rows, _vec

__all__ = ["group_norm_forward", "group_norm_backward", "Route", "route_forward", "route_backward", "conv_gate_backward"]


def _device(t, name):
    """The current device's number, on which `t` has to be."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device (cuda) tensor")
    return torch.cuda.current_device()


def _dense(t, name, dev, dtype, shape):
    """Checks a contiguous tensor (None passes); its address."""
    if t is None:
        return None
    _on(t, name, dev)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous of shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _group_sizes(x, groups, samples, activation, longest):
    """The leading arguments of a group norm's calls, x's row stride, number of samples,
    activation and device."""
    dev = _device(x, "x")
    ld = _rows(x, "x", dev)
    if activation not in ACT:
        raise ValueError(f"activation {activation!r}: one of {list(ACT)}")
    offsets, n = None, samples
    if isinstance(samples, torch.Tensor):
        _on(samples, "samples", dev)
        if samples.dtype is not torch.int32:
            raise TypeError(f"offsets of samples must be int32, got {samples.dtype}")
        if samples.dim() != 1 or samples.shape[0] < 1 or not samples.is_contiguous():
            raise ValueError(f"offsets of samples must be contiguous of shape (samples + 1,), got {tuple(samples.shape)}")
        offsets, n = samples.data_ptr(), samples.shape[0] - 1
    rows, width = x.shape
    return (ELEM[x.dtype], rows, width, groups, n, offsets, longest or 0), ld, n, ACT[activation], dev


def _group_room(backward, head, workspace, x):
    if workspace is None:
        b = ctypes.c_size_t()
        check(load().cgtp_group_norm_workspace_size(backward, *head, ctypes.byref(b)))
        if b.value:
            workspace = x.new_empty(b.value, dtype=torch.uint8)
    return workspace


def _pair(weight, bias, x, dev):
    """Addresses of weight and bias, and their type."""
    (w, tw), (b, tb) = _vec(weight, x.shape[1], "weight", x, dev), _vec(bias, x.shape[1], "bias", x, dev)
    if tw is not tb and tw is not None and tb is not None:
        raise TypeError(f"weight ({tw}) and bias ({tb}) must have one type")
    return w, b, tw or tb or torch.float32


def group_norm_forward(x, groups: int, weight=None, bias=None, samples=1, activation=None, eps: float = 1e-5, out=None,
                       longest: int | None = None, workspace=None):
    """y [rows, width] = activation(group norm of x) over each sample's rows and each group's
    columns, and stats [2, samples, groups] (mean and 1/sqrt(variance + eps), fp32) for the
    backward.

    x is fp32, bf16 or fp16, channels last: rows any stride apart.  samples: the number of
    samples of equal length, or an int32 device tensor [samples + 1] of their rows' bounds,
    ascending; rows before the first and behind the last belong to none: y is 0 there, or left
    as it is in a given `out`.  activation: None, "silu" or "gelu" (by erf).  weight and bias
    [width] are fp32 or x's type (None: 1, 0).  out: rows for y, any stride apart; x itself for
    a call in place, otherwise apart from x.  longest: rows of the longest sample, if they are
    known: with offsets on the device the call cannot see them, and chooses its launches by
    eight times the mean; it decides the speed only.  Asynchronous on the current stream;
    bitwise reproducible."""
    head, ld, n, act, dev = _group_sizes(x, groups, samples, activation, longest)
    w, b, wt = _pair(weight, bias, x, dev)
    zero = out is None
    if zero:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        ld_y = x.shape[1]
    else:
        ld_y = _rows(out, "out", dev, x.shape, x.dtype)
    workspace = _group_room(0, head, workspace, x)
    stats = x.new_empty((2, n, groups), dtype=torch.float32)
    check(load().cgtp_group_norm_forward(*head, x.data_ptr(), ld, ELEM[wt], w, b, act, eps, zero, out.data_ptr(), ld_y,
                                         stats.data_ptr(), *_room(workspace, dev), _raw_stream(dev)))
    return out, stats


def group_norm_backward(grad_out, x, stats, groups: int, weight=None, bias=None, samples=1, activation=None,
                        need=("x", "weight", "bias"), longest: int | None = None, workspace=None):
    """Gradients of a scalar L with dL/dy = grad_out: (grad_x [rows, width], grad_weight
    [width], grad_bias [width]); an entry not in `need` is None.  stats is the forward's, and
    weight, bias, samples and activation are as in its call.  grad_x is 0 for rows outside
    every sample.  grad_weight and grad_bias have weight's type (bias's, without a weight; fp32
    without both).  Asynchronous on the current stream; bitwise reproducible."""
    head, ld, n, act, dev = _group_sizes(x, groups, samples, activation, longest)
    ld_g = _rows(grad_out, "grad_out", dev, x.shape, x.dtype)
    w, b, wt = _pair(weight, bias, x, dev)
    st = _dense(stats, "stats", dev, torch.float32, (2, n, groups))
    if st is None:
        raise TypeError("stats must be a device (cuda) tensor")
    gx = torch.empty_like(x, memory_format=torch.contiguous_format) if "x" in need else None
    gw = x.new_empty(x.shape[1], dtype=wt) if "weight" in need else None
    gb = x.new_empty(x.shape[1], dtype=wt) if "bias" in need else None
    workspace = _group_room(1 if gw is not None or gb is not None else 2, head, workspace, x)
    check(load().cgtp_group_norm_backward(*head, grad_out.data_ptr(), ld_g, x.data_ptr(), ld, st, ELEM[wt], w, b, act,
                                          _at(gx), x.shape[1], _at(gw), _at(gb), *_room(workspace, dev),
                                          _raw_stream(dev)))
    return gx, gw, gb


class Route(NamedTuple):
    """What route_forward returns and route_backward takes."""
    ids: torch.Tensor       # [rows, k] int32, the largest logit's branch first, -1: none
    gates: torch.Tensor     # [rows, k] fp32; dense: [n, rows], 0 where not chosen
    counts: torch.Tensor    # [n] int32: rows that chose each branch
    balance: torch.Tensor   # [1] fp32: the balance loss
    slope: torch.Tensor     # [n] fp32: its derivative by each row's probabilities
    renormalise: bool
    dense: bool


def route_forward(logits, k: int, mask=None, renormalise: bool = False, dense: bool = False, workspace=None) -> Route:
    """Routes each row (edge) to the k of its n branches with the largest logits [rows, n].

    gates are the softmax probabilities of the chosen branches, divided by their sum if
    `renormalise`; with `dense`, gates[b] [rows] is the gate argument of branch b's conv_forward
    (a form for few branches: of more than 64 it is written one float at a time, slowly).
    balance = n sum over branches of (share of the choices) (mean probability): 1 where both are
    even, n where one branch has everything.  Rows with mask 0 (uint8 [rows]), or whose logits
    are all -inf, take no part; ties go to the lowest index.  logits are fp32, bf16 or fp16, rows
    any stride apart; n <= 1024, k <= 64.  Asynchronous on the current stream; bitwise
    reproducible."""
    dev = _device(logits, "logits")
    ld = _rows(logits, "logits", dev)
    rows, n = logits.shape
    at_mask = _dense(mask, "mask", dev, torch.uint8, (rows,))
    lib = load()
    if workspace is None:
        b = ctypes.c_size_t()
        check(lib.cgtp_route_workspace_size(rows, n, ctypes.byref(b)))
        workspace = logits.new_empty(b.value, dtype=torch.uint8) if b.value else None
    if not 1 <= k <= n:
        raise ValueError(f"{k} of {n} branches: need 1 <= k <= n")
    ids = logits.new_empty((rows, k), dtype=torch.int32)
    gates = logits.new_empty((n, rows) if dense else (rows, k), dtype=torch.float32)
    counts = logits.new_empty(n, dtype=torch.int32)
    balance, slope = logits.new_empty(1, dtype=torch.float32), logits.new_empty(n, dtype=torch.float32)
    check(lib.cgtp_route_forward(ELEM[logits.dtype], rows, n, k, logits.data_ptr(), ld, at_mask, renormalise, dense,
                                 ids.data_ptr(), gates.data_ptr(), counts.data_ptr(), balance.data_ptr(),
                                 slope.data_ptr(), *_room(workspace, dev), _raw_stream(dev)))
    return Route(ids, gates, counts, balance, slope, bool(renormalise), bool(dense))


def route_backward(logits, route: Route, grad_gates=None, grad_balance=None):
    """The logits' gradient [rows, n] (logits' type) of a scalar L: grad_gates = dL/dgates, laid
    out as route.gates (only entries of chosen branches are read), and grad_balance = dL/dbalance
    (fp32, one element, on the device); None stands for 0.  Choices and counts are held fixed.
    Asynchronous on the current stream; bitwise reproducible."""
    dev = _device(logits, "logits")
    ld = _rows(logits, "logits", dev)
    rows, n = logits.shape
    ids = route.ids
    k = ids.shape[1] if isinstance(ids, torch.Tensor) and ids.dim() == 2 else -1
    at_ids = _dense(ids, "route.ids", dev, torch.int32, (rows, k))
    slope = _dense(route.slope, "route.slope", dev, torch.float32, (n,))
    up = _dense(grad_gates, "grad_gates", dev, torch.float32, (n, rows) if route.dense else (rows, k))
    if grad_balance is not None:
        _on(grad_balance, "grad_balance", dev)
        if grad_balance.dtype is not torch.float32 or grad_balance.numel() != 1:
            raise TypeError("grad_balance must be a float32 tensor of one element")
    grad = torch.empty_like(logits, memory_format=torch.contiguous_format)
    check(load().cgtp_route_backward(ELEM[logits.dtype], rows, n, k, logits.data_ptr(), ld, route.renormalise,
                                     route.dense, at_ids, slope, up, _at(grad_balance), grad.data_ptr(), n,
                                     _raw_stream(dev)))
    return grad


def conv_gate_backward(w, grad_w, gate, mask=None, out=None):
    """dL/dgate [E] of the convolution's gate, from its weights w [E, W] and their gradient
    grad_w that conv_backward gave with that gate (and mask): sum of w grad_w / gate, 0 for
    inactive edges, whose rows are not read.  fp32.  out: [E] to write into.  Asynchronous on
    the current stream; bitwise reproducible."""
    dev = _device(w, "w")
    if w.dim() != 2:
        raise ValueError(f"w has shape {tuple(w.shape)}, expected (edges, weights)")
    at_w = _dense(w, "w", dev, torch.float32, w.shape)
    if grad_w is None or gate is None:
        raise TypeError("grad_w and gate must be device (cuda) tensors")
    at_g = _dense(grad_w, "grad_w", dev, torch.float32, w.shape)
    edges, width = w.shape
    at_gate, at_mask = _dense(gate, "gate", dev, torch.float32, (edges,)), _dense(mask, "mask", dev, torch.uint8, (edges,))
    if out is None:
        out = torch.empty_like(gate)
    check(load().cgtp_conv_gate_backward(edges, width, at_w, at_g, at_mask, at_gate,
                                         _dense(out, "out", dev, torch.float32, (edges,)), _raw_stream(dev)))
    return out
