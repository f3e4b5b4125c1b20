"""Plain fp64 references of the operators for branching networks: group normalisation with
an activation, routing with its balance loss, the gradient of the convolution's gate.

Written from the definitions that include/cgtp.h states, in numpy, sharing no code with
the HIP path.  Pinned by tests/test_oracle_branch.py: the normalisation by the plain
definition of standardised groups and central differences; the routing by a loop over rows,
by its closed forms for even and for one-sided choices, and by central differences; the
gate's gradient by central differences of the convolution.
"""
from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(z, act):
    """(act(z), act'(z))."""
    if act == "silu":
        with np.errstate(over="ignore"):
            p = 1 / (1 + np.exp(-z))
        return z * p, p + z * p * (1 - p)
    if act == "gelu":
        p = 0.5 * (1 + _erf(z / math.sqrt(2)))
        return z * p, p + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return z, np.ones_like(z)


def _blocks(x, offsets, groups):
    """(sample, group, rows, columns) of each sample that has rows."""
    c = x.shape[1] // groups
    for s, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        if hi > lo:
            for g in range(groups):
                yield s, g, slice(lo, hi), slice(g * c, (g + 1) * c)


def group_norm_forward(x, groups, offsets, weight=None, bias=None, act=None, eps=1e-5):
    """(y, mean [samples, groups], rstd); y is 0 in rows outside every sample."""
    x = np.asarray(x, dtype=np.float64)
    w = np.ones(x.shape[1]) if weight is None else np.asarray(weight, dtype=np.float64)
    b = np.zeros(x.shape[1]) if bias is None else np.asarray(bias, dtype=np.float64)
    n = len(offsets) - 1
    y, mean, rstd = np.zeros_like(x), np.zeros((n, groups)), np.full((n, groups), 1 / np.sqrt(eps) if eps else np.inf)
    for s, g, r, c in _blocks(x, offsets, groups):
        mean[s, g] = x[r, c].mean()
        rstd[s, g] = 1 / np.sqrt(((x[r, c] - mean[s, g]) ** 2).mean() + eps)
        y[r, c] = activation((x[r, c] - mean[s, g]) * rstd[s, g] * w[c] + b[c], act)[0]
    return y, mean, rstd


def group_norm_backward(grad_out, x, groups, offsets, weight=None, bias=None, act=None, eps=1e-5):
    """(grad_x, grad_weight, grad_bias) with the statistics of x itself."""
    x, go = np.asarray(x, dtype=np.float64), np.asarray(grad_out, dtype=np.float64)
    w = np.ones(x.shape[1]) if weight is None else np.asarray(weight, dtype=np.float64)
    b = np.zeros(x.shape[1]) if bias is None else np.asarray(bias, dtype=np.float64)
    _, mean, rstd = group_norm_forward(x, groups, offsets, eps=eps)
    gx, gw, gb = np.zeros_like(x), np.zeros(x.shape[1]), np.zeros(x.shape[1])
    for s, g, r, c in _blocks(x, offsets, groups):
        h = (x[r, c] - mean[s, g]) * rstd[s, g]
        d = go[r, c] * activation(h * w[c] + b[c], act)[1]
        a = d * w[c]
        gx[r, c] = rstd[s, g] * (a - a.mean() - h * (a * h).mean())
        gw[c] += (d * h).sum(axis=0)
        gb[c] += d.sum(axis=0)
    return gx, gw, gb


def softmax(z):
    z = np.asarray(z, dtype=np.float64)
    top = z.max(axis=1, keepdims=True)
    e = np.exp(z - np.where(np.isfinite(top), top, 0.0))
    s = e.sum(axis=1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def route_forward(logits, k, mask=None, renormalise=False):
    """(ids [rows, k], gates [rows, k], counts [n], balance, slope [n]) of finite or -inf logits."""
    z = np.asarray(logits, dtype=np.float64)
    rows, n = z.shape
    part = (z > -np.inf).any(axis=1)
    if mask is not None:
        part &= np.asarray(mask) != 0
    p = softmax(z) * part[:, None]
    ids = np.argsort(-z, axis=1, kind="stable")[:, :k]
    some = np.take_along_axis(z, ids, axis=1) > -np.inf
    some &= part[:, None]
    gates = np.take_along_axis(p, ids, axis=1) * some
    if renormalise:
        total = gates.sum(axis=1, keepdims=True)
        gates = np.divide(gates, total, out=np.zeros_like(gates), where=total > 0)
    ids = np.where(some, ids, -1)
    counts = np.array([(ids == e).sum() for e in range(n)])
    both = float(counts.sum()) * float(part.sum())
    slope = n * counts / both if both else np.zeros(n)
    return ids, gates, counts, float((slope * p.sum(axis=0)).sum()), slope


def dense_gates(ids, gates, n):
    """[rows, k] as [n, rows]."""
    out = np.zeros((n, ids.shape[0]))
    for i in range(ids.shape[1]):
        r = np.nonzero(ids[:, i] >= 0)[0]
        out[ids[r, i], r] = gates[r, i]
    return out


def route_backward(logits, ids, slope, grad_gates=None, grad_balance=0.0, renormalise=False):
    """Gradient of sum(grad_gates gates) + grad_balance balance, choices and slope held fixed."""
    z = np.asarray(logits, dtype=np.float64)
    p = softmax(z)
    up, take = np.zeros_like(p), np.zeros_like(p)
    for i in range(ids.shape[1]):
        r = np.nonzero(ids[:, i] >= 0)[0]
        take[r, ids[r, i]] = 1
        if grad_gates is not None:
            up[r, ids[r, i]] = np.asarray(grad_gates, dtype=np.float64)[r, i]
    u = np.broadcast_to(grad_balance * np.asarray(slope, dtype=np.float64), p.shape)
    if renormalise:
        total = (p * take).sum(axis=1, keepdims=True)
        q = np.divide(p * take, total, out=np.zeros_like(p), where=total > 0)
        extra = q * (up - (up * q).sum(axis=1, keepdims=True))
    else:
        u, extra = u + up, 0.0
    grad = p * (u - (u * p).sum(axis=1, keepdims=True)) + extra
    return grad * (ids[:, :1] >= 0)


def gate_backward(w, grad_w, gate, mask=None):
    w, g, f = (np.asarray(v, dtype=np.float64) for v in (w, grad_w, gate))
    on = f != 0
    if mask is not None:
        on &= np.asarray(mask) != 0
    out = np.zeros(len(f))
    out[on] = (w[on] * g[on]).sum(axis=1) / f[on]
    return out
