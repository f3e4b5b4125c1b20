"""Operators that train a network around the convolution: layer normalisation of rows,
its equivariant form over irreps, and the AdamW step over many tensors with 32-bit or
8-bit moments and a gradient norm.

Argument marshalling over libcgtp.so as in the package's other calls: device tensors in,
the HIP kernels on the caller's current torch stream, no fallback.  Like conv_forward they
stand outside autograd: results carry no history.  examples/train_potential.py wraps them in
torch.autograd.Function; there are no second derivatives.  The formulas stand in
include/cgtp.h beside each entry point.

    y, stats = layer_norm_forward(hidden, gamma, beta)
    grad_hidden, grad_gamma, grad_beta = layer_norm_backward(grad_y, hidden, stats, gamma)

    norm = NormPlan(plan.irreps_out)
    y, stats = irreps_norm_forward(norm, out, weight, bias)

    params = ParamSet([p.numel() for p in tensors], weight_decay=0.01)
    state = adamw_state(params, bits=8)
    factor = grad_norm(params, grads, max_norm=1.0)[1:]
    adamw_step(params, tensors, grads, state, lr=1e-3, step=t, grad_scale=factor, seed=t)
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import ELEM, check, load

__all__ = ["layer_norm_forward", "layer_norm_backward", "NormPlan", "irreps_norm_forward", "irreps_norm_backward",
           "ParamSet", "adamw_state", "adamw_step", "adamw_moments", "grad_norm"]


def _raw_stream(device):
    return torch.cuda.current_stream(device).cuda_stream


# current_stream() makes an object, 3 us a call.  A torch without devices lacks the other name
# and calls neither.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _on(t, name, dev):
    """Checks that t is a tensor on device number `dev`."""
    at = t.get_device() if isinstance(t, torch.Tensor) else -1   # -1: on the host
    if at != dev:
        if at < 0:
            raise TypeError(f"{name} must be a device (cuda) tensor")
        raise ValueError(f"{name} is on device {at}, expected {dev}")


def _rows(t, name, dev, shape=None, dtype=None):
    """Checks a [rows, width] tensor on device `dev` whose rows are dense; its row stride."""
    _on(t, name, dev)
    if (t.dtype is not dtype) if dtype is not None else (t.dtype not in ELEM):
        raise TypeError(f"{name} must be {dtype or 'float32, bfloat16 or float16'}, got {t.dtype}")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {'(rows, width)' if shape is None else tuple(shape)}")
    n, f = t.shape
    ld, inner = t.stride()
    if (inner != 1 and f > 1) or (ld < f and n > 1):
        raise ValueError(f"{name} must have dense rows that do not overlap, got strides {t.stride()}")
    return ld if ld > f else f


def _vec(t, n, name, x, dev):
    """Checks a weight or bias [n] of fp32 or x's type (None passes); its address and type."""
    if t is None:
        return None, None
    _on(t, name, dev)
    d = t.dtype
    if d is not torch.float32 and d is not x.dtype:
        raise TypeError(f"{name} must be float32 or {x.dtype}, got {d}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous of shape ({n},), got {tuple(t.shape)}")
    return t.data_ptr(), d


def _head(plan, x):
    """The leading arguments of a norm call, and x's row stride, weights, biases, shape of
    stats and device.  The library's calls run on the current device: x has to be there."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("x must be a device (cuda) tensor")
    dev = torch.cuda.current_device()
    ld = _rows(x, "x", dev)
    n, f = x.shape
    if plan is None:
        return (ELEM[x.dtype], n, f), ld, f, f, (2, n), dev
    if f != plan.n_features:
        raise ValueError(f"x has rows of {f}, the plan's have {plan.n_features}")
    return (plan.handle, ELEM[x.dtype], n), ld, plan.n_weights, plan.n_biases, (2, n, plan.n_terms), dev


def _forward(call, plan, x, weight, bias, eps, out):
    head, ld, nw, nb, stats_shape, dev = _head(plan, x)
    (w, tw), (b, tb) = _vec(weight, nw, "weight", x, dev), _vec(bias, nb, "bias", x, dev)
    if tw is not tb and tw is not None and tb is not None:
        raise TypeError(f"weight ({tw}) and bias ({tb}) must have one type")
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        ld_y = x.shape[1]
    else:
        ld_y = _rows(out, "out", dev, x.shape, x.dtype)
    stats = x.new_empty(stats_shape, dtype=torch.float32)
    check(call(*head, x.data_ptr(), ld, ELEM[tw or tb or torch.float32], w, b, eps, out.data_ptr(), ld_y,
               stats.data_ptr(), _raw_stream(dev)))
    return out, stats


def _backward(call, size, plan, grad_out, x, stats, weight, need, workspace):
    head, ld, nw, nb, stats_shape, dev = _head(plan, x)
    ld_g = _rows(grad_out, "grad_out", dev, x.shape, x.dtype)
    w, wt = _vec(weight, nw, "weight", x, dev)
    wt = wt or torch.float32
    _on(stats, "stats", dev)
    if stats.dtype != torch.float32:
        raise TypeError(f"stats must be float32, got {stats.dtype}")
    if stats.shape != stats_shape or not stats.is_contiguous():
        raise ValueError(f"stats must be contiguous of shape {stats_shape}, got {tuple(stats.shape)}")
    gx = torch.empty_like(x, memory_format=torch.contiguous_format) if "x" in need else None
    gw = x.new_empty(nw, dtype=wt) if "weight" in need else None
    gb = x.new_empty(nb, dtype=wt) if "bias" in need else None
    if workspace is None and (gw is not None or gb is not None):
        need_bytes = size(x.shape[0])
        workspace = x.new_empty(need_bytes, dtype=torch.uint8) if need_bytes else None
    check(call(*head, grad_out.data_ptr(), ld_g, x.data_ptr(), ld, stats.data_ptr(), ELEM[wt], w, _at(gx), x.shape[1],
               _at(gw), _at(gb), *_room(workspace, dev), _raw_stream(dev)))
    return gx, gw, gb


def _at(t):
    return None if t is None else t.data_ptr()


def _room(workspace, dev):
    """Checks a workspace (may be None); its address and bytes."""
    if workspace is None:
        return None, 0
    _on(workspace, "workspace", dev)
    if not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous, got strides {workspace.stride()}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def layer_norm_forward(x, weight=None, bias=None, eps: float = 1e-5, out=None):
    """y [rows, width] of the layer norm of each row of x, and stats [2, rows] (mean and
    1/sqrt(variance + eps), fp32) for the backward.

    x is fp32, bf16 or fp16 with dense rows any stride apart; weight and bias [width] are
    fp32 or x's type (None: 1, 0).  out: rows for y, any stride apart; x itself for a call in
    place, otherwise apart from x.  Asynchronous on the current stream."""
    return _forward(load().cgtp_layer_norm_forward, None, x, weight, bias, eps, out)


def layer_norm_backward(grad_out, x, stats, weight=None, need=("x", "weight", "bias"), workspace=None):
    """Gradients of a scalar L with dL/dy = grad_out: (grad_x [rows, width], grad_weight
    [width], grad_bias [width]); an entry not in `need` is None.  stats is the forward's.
    grad_weight and grad_bias have weight's type (fp32 without one).  Asynchronous on the
    current stream; bitwise reproducible."""
    lib = load()

    def size(n):
        b = ctypes.c_size_t()
        check(lib.cgtp_layer_norm_backward_workspace_size(n, x.shape[1], ctypes.byref(b)))
        return b.value

    return _backward(lib.cgtp_layer_norm_backward, size, None, grad_out, x, stats, weight, need, workspace)


class NormPlan:
    """The equivariant layer norm of irreps rows ("128x0e+64x1o"): each term by itself,
    0e terms centred and with a bias, every channel with a weight."""

    def __init__(self, irreps: str):
        lib = load()
        h = ctypes.c_void_p()
        check(lib.cgtp_norm_create(irreps.encode(), ctypes.byref(h)))
        self._h = h
        f, w, b, t = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int()
        check(lib.cgtp_norm_info(h, ctypes.byref(f), ctypes.byref(w), ctypes.byref(b), ctypes.byref(t)))
        self.irreps = irreps
        self.n_features, self.n_weights, self.n_biases, self.n_terms = f.value, w.value, b.value, t.value

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("plan is closed")
        return self._h

    def backward_workspace_size(self, n_rows: int) -> int:
        b = ctypes.c_size_t()
        check(load().cgtp_irreps_norm_backward_workspace_size(self.handle, int(n_rows), ctypes.byref(b)))
        return b.value

    def close(self):
        if getattr(self, "_h", None) is not None:
            load().cgtp_norm_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def irreps_norm_forward(plan: NormPlan, x, weight=None, bias=None, eps: float = 1e-5, out=None):
    """y [rows, plan.n_features] and stats [2, rows, plan.n_terms]; weight
    [plan.n_weights] one per channel, bias [plan.n_biases] one per 0e channel.  Types and
    strides as layer_norm_forward."""
    return _forward(load().cgtp_irreps_norm_forward, plan, x, weight, bias, eps, out)


def irreps_norm_backward(plan: NormPlan, grad_out, x, stats, weight=None, need=("x", "weight", "bias"),
                         workspace=None):
    """(grad_x, grad_weight [plan.n_weights], grad_bias [plan.n_biases]) as
    layer_norm_backward."""
    return _backward(load().cgtp_irreps_norm_backward, plan.backward_workspace_size, plan, grad_out, x, stats, weight,
                     need, workspace)


class _Pointers:
    """Device pointers of a set's tensors, checked and laid out for the library; keeps the
    tensors and the memory that they have now alive."""

    def __init__(self, tensors, sizes):
        tensors = list(tensors)
        if len(tensors) != len(sizes):
            raise ValueError(f"{len(tensors)} tensors, the set has {len(sizes)}")
        for k, (t, n) in enumerate(zip(tensors, sizes)):
            at = t.get_device() if isinstance(t, torch.Tensor) else -1
            if at < 0:
                raise TypeError(f"tensor {k} must be a device (cuda) tensor")
            if k == 0:
                dev, dtype = at, t.dtype
            if t.dtype is not dtype or dtype not in ELEM:
                raise TypeError(f"tensor {k} is {t.dtype}: one type, float32, bfloat16 or float16")
            if at != dev:
                raise ValueError("the tensors of a set are on one device")
            if t.numel() != n:
                raise ValueError(f"tensor {k} has {t.numel()} elements, expected {n}")
            if not t.is_contiguous():
                raise ValueError(f"tensor {k} must be contiguous")
        self.tensors, self.sizes = tensors, sizes
        self.device = tensors[0].device if tensors else None
        self.type = ELEM[tensors[0].dtype] if tensors else 0
        addresses = [t.data_ptr() for t in tensors]
        self.array = (ctypes.c_void_p * max(len(tensors), 1))(*addresses)
        # a tensor that is given other memory would free what the addresses name: 50 ns each
        self.storages = list(map(torch.Tensor.untyped_storage, tensors))
        # looked at by every call; all tensors, at 40 ns each, would make a step of 96 21 us for 15
        self.ends = [(tensors[k].data_ptr, addresses[k]) for k in (0, -1)] if tensors else []

    def moved(self):
        """Whether the first or the last tensor has other memory now."""
        for address, at in self.ends:
            if address() != at:
                return True
        return False


class ParamSet:
    """The tensors that one optimiser step covers: their sizes (ints, or tensors whose
    numel is taken) and weight decay (one number, or one per tensor).  Device tables are on
    the device that is current when it is made (host_only: none, sizes only)."""

    def __init__(self, sizes, weight_decay=0.0, host_only: bool = False):
        lib = load()
        self.sizes = [int(s.numel()) if isinstance(s, torch.Tensor) else int(s) for s in sizes]
        n = len(self.sizes)
        decay = list(weight_decay) if hasattr(weight_decay, "__iter__") else [weight_decay] * n
        if len(decay) != n:
            raise ValueError(f"{len(decay)} weight decays for {n} tensors")
        h = ctypes.c_void_p()
        check(lib.cgtp_params_create((ctypes.c_int64 * max(n, 1))(*self.sizes), (ctypes.c_double * max(n, 1))(*decay),
                                     n, _lib.CGTP_PLAN_HOST_ONLY if host_only else 0, ctypes.byref(h)))
        self._h = h
        elems, offs = ctypes.c_int64(), (ctypes.c_int64 * max(n, 1))()
        check(lib.cgtp_params_info(h, None, ctypes.byref(elems), offs))
        self.state_elems, self.offsets = elems.value, list(offs)[:n]
        b = ctypes.c_size_t()
        check(lib.cgtp_grad_norm_workspace_size(h, ctypes.byref(b)))
        self.grad_norm_workspace_size = b.value
        self.index = None if host_only else torch.cuda.current_device()
        self.device = None if host_only else torch.device("cuda", self.index)

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("set is closed")
        return self._h

    def pointers(self, tensors) -> _Pointers:
        """The set's parameters or gradients laid out once, for calls that use the same
        tensors again; the calls also take the plain list, and lay it out each time.

        A layout is of the memory that the tensors have when it is made, and keeps it alive.
        Lay them out again after any of them is given other memory (t.data = ..., set_,
        Module.to): calls would go on with the old one.  They refuse a layout whose first or
        last tensor has moved, as all do in Module.to, and do not look at the others.  A
        storage that is resized in place frees its memory all the same: lay out again before
        the next call."""
        return tensors if isinstance(tensors, _Pointers) else _Pointers(tensors, self.sizes)

    def close(self):
        if getattr(self, "_h", None) is not None:
            load().cgtp_params_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def adamw_state(params: ParamSet, bits: int = 32):
    """Zeroed states of a set: (m, v) fp32, or with bits=8 (m codes, r codes, m exponents,
    r exponents), uint8, of m and r = sqrt(v).  Tensor t's begin at params.offsets[t]."""
    n = params.state_elems
    if bits == 32:
        return tuple(torch.zeros(n, dtype=torch.float32, device=params.device) for _ in range(2))
    if bits == 8:
        return tuple(torch.zeros(k, dtype=torch.uint8, device=params.device) for k in (n, n, n // 64, n // 64))
    raise ValueError("states have 32 or 8 bits")


def _state(params, state):
    """Checks a set's states; their addresses."""
    if len(state) not in (2, 4):
        raise ValueError("a state is (m, v) or (m codes, r codes, m exponents, r exponents)")
    dtype = torch.float32 if len(state) == 2 else torch.uint8
    dev, n, at = params.index, params.state_elems, []
    for k, t in enumerate(state):
        _on(t, "a state", dev)
        if t.dtype != dtype:
            raise TypeError(f"a state is {t.dtype}, expected {dtype}")
        if k == 2:
            n //= 64
        if t.numel() != n or t.dim() != 1 or not t.is_contiguous():
            raise ValueError(f"a state has shape {tuple(t.shape)}, expected ({n},), contiguous")
        at.append(t.data_ptr())
    return at


def _scale(params, t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != params.index or t.dtype != torch.float32 or t.numel() != 1:
        raise TypeError("grad_scale must be a float32 tensor of one element on the set's device")
    return t.data_ptr()


def _laid(params, tensors, what):
    p = params.pointers(tensors)
    if p.sizes is not params.sizes and p.sizes != params.sizes:
        raise ValueError(f"{what} were laid out for another set")
    if p.device is not None and p.device != params.device:
        raise ValueError(f"{what} must be on the set's device")
    if p is tensors and p.moved():
        raise ValueError(f"{what} have other memory than when they were laid out: lay them out again")
    return p


def _scalars(params, lr, betas, step, scale, seed, stream):
    """The scalars of a step that is counted on the device; the tensor that holds them."""
    if step.get_device() != params.index or step.dtype != torch.int64 or step.numel() != 1:
        raise TypeError("step must be an int, or an int64 tensor of one element on the set's device")
    lr_at = None
    if isinstance(lr, torch.Tensor):
        if lr.get_device() != params.index or lr.dtype != torch.float32 or lr.numel() != 1:
            raise TypeError("lr must be a number, or a float32 tensor of one element on the set's device")
        lr, lr_at = 0.0, lr.data_ptr()
    out = torch.empty(_lib.CGTP_ADAMW_SCALARS_BYTES // 8, dtype=torch.int64, device=params.device)
    check(load().cgtp_adamw_scalars(step.data_ptr(), lr_at, lr, betas[0], betas[1], seed & 0xffffffff, scale,
                                    out.data_ptr(), stream))
    return out


def adamw_step(params: ParamSet, tensors, grads, state, lr, betas=(0.9, 0.999), eps: float = 1e-8, step=1,
               grad_scale=None, seed: int = 0):
    """One AdamW step of the set, in place on `tensors` and `state`; step counts from 1.

    tensors and grads: lists of contiguous device tensors (or params.pointers of them).
    grad_scale: a device tensor of one fp32 (grad_norm's second value, or an inverse loss
    scale) that multiplies the gradients; NaN skips the step.  With 8-bit states, seed
    chooses the rounding: pass another each step.  Asynchronous on the current stream.

    For steps in a captured graph, step is an int64 device tensor of one element, 0 before
    the first step: the call advances it (unless the step is skipped), and adds its number
    to the seed.  lr may then be a device tensor of one fp32."""
    p, g = _laid(params, tensors, "tensors"), _laid(params, grads, "grads")
    s, scale, stream = _state(params, state), _scale(params, grad_scale), _raw_stream(params.index)
    lib, at = load(), None
    if isinstance(step, torch.Tensor):
        scalars = _scalars(params, lr, betas, step, scale, seed, stream)
        lr, step, at = 0.0, 1, scalars.data_ptr()
    if len(s) == 2:
        check(lib.cgtp_adamw_step(params.handle, p.type, p.array, g.type, g.array, *s, lr, betas[0], betas[1], eps,
                                  step, at, scale, stream))
    else:
        check(lib.cgtp_adamw_step_8bit(params.handle, p.type, p.array, g.type, g.array, *s, lr, betas[0], betas[1],
                                       eps, step, seed & 0xffffffff, at, scale, stream))


def adamw_moments(params: ParamSet, state):
    """The values of 8-bit states: m and r = sqrt(v) [state_elems], in bf16, which holds
    them exactly; 32-bit states are returned as they are."""
    s = _state(params, state)
    if len(s) == 2:
        return state
    m, r = (torch.empty(params.state_elems, dtype=torch.bfloat16, device=params.device) for _ in range(2))
    check(load().cgtp_adamw_read_8bit(params.handle, *s, m.data_ptr(), r.data_ptr(),
                                      _raw_stream(params.index)))
    return m, r


def grad_norm(params: ParamSet, grads, max_norm: float = float("inf"), grad_scale=None, workspace=None):
    """[2] fp32 on the device: the 2-norm of all gradients (times grad_scale) and the
    factor grad_scale min(1, max_norm / norm) for adamw_step, NaN where the norm is not
    finite.  Asynchronous on the current stream; bitwise reproducible."""
    g = _laid(params, grads, "grads")
    out = torch.empty(2, dtype=torch.float32, device=params.device)
    if workspace is None and params.grad_norm_workspace_size:
        workspace = torch.empty(params.grad_norm_workspace_size, dtype=torch.uint8, device=params.device)
    check(load().cgtp_grad_norm(params.handle, g.type, g.array, _scale(params, grad_scale), max_norm, out.data_ptr(),
                                *_room(workspace, params.index), _raw_stream(params.index)))
    return out
