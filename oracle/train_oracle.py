"""Plain fp64 references of the training operators: layer normalisation of rows and of
irreps rows, AdamW with 32-bit and 8-bit moments, the gradient norm.

Written from the definitions that include/cgtp.h states, in numpy, sharing no code with
the HIP path.  Pinned by tests/test_oracle_train.py: the normalisations by central
differences, by rotation and inversion equivariance and by the plain definition of a
standardised row; AdamW by its closed form for a constant gradient; the 8-bit codec by
its grid, its rounding's mean and the uniformity of its hash.
"""
from __future__ import annotations

import numpy as np

from .cgtp_oracle import parse_irreps

BLOCK = 64


def norm_terms(irreps: str):
    """(offset, channels, components, first weight, first bias or None) of each term."""
    out, off, w, b = [], 0, 0, 0
    for mul, l, p in parse_irreps(irreps):
        centred = l == 0 and p == 1
        out.append((off, mul, 2 * l + 1, w, b if centred else None))
        off, w, b = off + mul * (2 * l + 1), w + mul, b + (mul if centred else 0)
    return out


def row_terms(width: int):
    """The one term of a plain layer norm."""
    return [(0, width, 1, 0, 0)]


def norm_forward(x, terms, weight=None, bias=None, eps=1e-5):
    """(y, mean [rows, terms], rstd [rows, terms])."""
    x = np.asarray(x, dtype=np.float64)
    n = x.shape[0]
    y, mean, rstd = np.zeros_like(x), np.zeros((n, len(terms))), np.zeros((n, len(terms)))
    for k, (off, mul, d, w0, b0) in enumerate(terms):
        q = x[:, off:off + mul * d].reshape(n, mul, d)
        if b0 is not None:
            mean[:, k] = q.mean(axis=(1, 2))
        c = q - mean[:, k, None, None]
        rstd[:, k] = 1 / np.sqrt((c ** 2).mean(axis=(1, 2)) + eps)
        h = c * rstd[:, k, None, None]
        if weight is not None:
            h = h * np.asarray(weight, dtype=np.float64)[None, w0:w0 + mul, None]
        if bias is not None and b0 is not None:
            h = h + np.asarray(bias, dtype=np.float64)[None, b0:b0 + mul, None]
        y[:, off:off + mul * d] = h.reshape(n, -1)
    return y, mean, rstd


def norm_backward(grad_out, x, terms, weight=None, eps=1e-5):
    """(grad_x, grad_weight, grad_bias) with the statistics of x itself."""
    x, g = np.asarray(x, dtype=np.float64), np.asarray(grad_out, dtype=np.float64)
    n = x.shape[0]
    _, mean, rstd = norm_forward(x, terms, eps=eps)
    gx = np.zeros_like(x)
    gw = np.zeros(sum(t[1] for t in terms))
    gb = np.zeros(sum(t[1] for t in terms if t[4] is not None))
    for k, (off, mul, d, w0, b0) in enumerate(terms):
        sl = slice(off, off + mul * d)
        r = rstd[:, k, None, None]
        h = (x[:, sl].reshape(n, mul, d) - mean[:, k, None, None]) * r
        go = g[:, sl].reshape(n, mul, d)
        a = go if weight is None else go * np.asarray(weight, dtype=np.float64)[None, w0:w0 + mul, None]
        v = a - h * (a * h).mean(axis=(1, 2), keepdims=True)
        if b0 is not None:
            v = v - a.mean(axis=(1, 2), keepdims=True)
            gb[b0:b0 + mul] = go.sum(axis=(0, 2))
        gx[:, sl] = (v * r).reshape(n, -1)
        gw[w0:w0 + mul] = (go * h).sum(axis=(0, 2))
    return gx, gw, gb


def adamw(p, g, m, v, lr, beta1, beta2, eps, step, decay=0.0, scale=1.0):
    """(p, m, v) after one step, in fp64."""
    p, g, m, v = (np.asarray(q, dtype=np.float64) for q in (p, g, m, v))
    g = g * scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mh, vh = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return p - lr * decay * p - lr * mh / (np.sqrt(vh) + eps), m, v


def adamw_f32(p, g, m, v, lr, beta1, beta2, eps, step, decay=0.0, scale=1.0):
    """(p, m, v, sqrt(v)) after one step computed as documented: every operation one fp32
    rounding, in the stated order."""
    f = np.float32
    with np.errstate(all="ignore"):
        g = np.asarray(g, dtype=f) * f(scale)
        p = np.asarray(p, dtype=f) * f(1 - float(lr) * float(decay))
        m = np.asarray(m, dtype=f) * f(beta1) + g * f(1 - beta1)
        v = np.asarray(v, dtype=f) * f(beta2) + g * g * f(1 - beta2)
        root = np.sqrt(v)
        p = p - m * f(lr / (1 - beta1 ** step)) / (root * f(1 / np.sqrt(1 - beta2 ** step)) + f(eps))
    return p, m, v, root


def random_bits(i, seed):
    """The 32 bits of the stochastic rounding of state elements i."""
    i = np.asarray(i, dtype=np.uint64)
    with np.errstate(over="ignore"):
        h = (i.astype(np.uint32) * np.uint32(0x9E3779B9) + (i >> np.uint64(32)).astype(np.uint32) * np.uint32(0x6A09E667)
             + np.uint32((seed * 0x3C6EF373) & 0xffffffff))
        h ^= h >> np.uint32(15)
        h *= np.uint32(0xBB67AE85)
        return h ^ (h >> np.uint32(16))


def _grid(code, mantissa):
    """Value of magnitude codes in units of 2^(exponent byte - 127)."""
    x, f = code >> mantissa, code & ((1 << mantissa) - 1)
    return np.where(x > 0, f + (1 << mantissa), f) * 2.0 ** (np.maximum(x, 1) - 14 - mantissa)


def decode(code, exponent, signed):
    """fp64 values of uint8 codes [n] with exponent bytes [n / 64]."""
    code = np.asarray(code).astype(np.int64)
    scale = 2.0 ** (np.maximum(np.repeat(np.asarray(exponent).astype(np.int64), BLOCK), 1) - 127)
    if signed:
        mag = code & 127
        val = np.where(mag == 127, np.nan, _grid(mag, 3) * scale)
        return np.where(code > 127, -val, val)
    return np.where(code == 255, np.nan, _grid(code, 4) * scale)


def encode(value, u, signed):
    """(codes, exponent bytes) of fp32 values [n] with 16 random bits u each: by search on
    the grid of decode()."""
    v = np.asarray(value, dtype=np.float32)
    mant, top = (3, 127) if signed else (4, 255)
    a = np.abs(v.astype(np.float64))
    fine = np.isfinite(a)
    a = np.where(fine, a, 0.0)
    e = (np.abs(v).view(np.uint32) >> 23).astype(np.int64)
    e = np.where(fine, e, 0).reshape(-1, BLOCK).max(axis=1)
    unit = np.repeat(2.0 ** (np.maximum(e, 1) - 127), BLOCK)
    grid = _grid(np.arange(top), mant)
    q = a / unit
    lo = np.searchsorted(grid, q, side="right") - 1
    frac = (q - grid[lo]) / (grid[np.minimum(lo + 1, top - 1)] - grid[lo])
    code = lo + (frac + np.asarray(u) / 65536.0 >= 1)
    if signed:
        code = np.where(fine, code, 127) | np.where(v < 0, 128, 0)
    else:
        code = np.where((a > 0) & (code == 0), 1, code)
        code = np.where(fine, code, 255)
    return code.astype(np.uint8), e.astype(np.uint8)


def grad_norm(grads, scale=1.0, max_norm=np.inf):
    """(norm, factor)."""
    s = np.sqrt(sum(float((np.asarray(g, dtype=np.float64) ** 2).sum()) for g in grads)) * abs(scale)
    if not np.isfinite(s):
        return s, np.nan
    return s, scale * min(1.0, max_norm / s) if s > 0 else scale
