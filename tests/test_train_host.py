"""CPU checks of the training operators' entry points: plan and set bookkeeping and every
refusal that happens on the host before a launch.  No device work is done here."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import train_oracle as T

C = pytest.importorskip("clebsch_gordan_tensor_node_amd")

INVALID, PARSE, UNSUPPORTED, WORKSPACE = -1, -2, -3, -5
F32, BF16, F16 = 0, 1, 2


def _ptr(a):
    return ctypes.c_void_p(a.ctypes.data)


@pytest.mark.parametrize("irreps", ["8x0e", "16x0e+8x1e+16x1o", "3x0o+2x0e+1x6e+5x0e", "1o"])
def test_norm_plan_counts(irreps):
    p, t = C.NormPlan(irreps), T.norm_terms(irreps)
    assert p.n_features == sum(m * d for _, m, d, _, _ in t) and p.n_weights == sum(m for _, m, _, _, _ in t)
    assert p.n_biases == sum(m for _, m, _, _, b in t if b is not None) and p.n_terms == len(t)
    p.close()
    with pytest.raises(ValueError):
        p.handle


@pytest.mark.parametrize("irreps,code", [("", PARSE), ("8x", PARSE), ("4x0q", PARSE), ("4x7e", UNSUPPORTED),
                                         ("0x1e", UNSUPPORTED), ("+".join(["1x0e"] * 65), UNSUPPORTED),
                                         ("999999999x6e", UNSUPPORTED)])
def test_norm_plan_refusals(irreps, code):
    with pytest.raises(C.CgtpError) as e:
        C.NormPlan(irreps)
    assert e.value.code == code


def test_param_set_offsets():
    s = C.ParamSet([1, 0, 64, 65, 4097], [0, 0, 0.1, 0, 0], host_only=True)
    assert s.offsets == [0, 64, 64, 128, 256] and s.state_elems == 256 + 4160
    assert C.ParamSet([], host_only=True).state_elems == 0
    assert C.ParamSet([torch.zeros(3, 5)], host_only=True).sizes == [15]


@pytest.mark.parametrize("sizes,decay,code", [([-1], [0.0], INVALID), ([4], [-0.1], INVALID), ([4], [np.nan], INVALID),
                                              ([1 << 41], [0.0], UNSUPPORTED)])
def test_param_set_refusals(sizes, decay, code):
    with pytest.raises(C.CgtpError) as e:
        C.ParamSet(sizes, decay, host_only=True)
    assert e.value.code == code
    with pytest.raises(ValueError):
        C.ParamSet([1, 2], [0.0], host_only=True)


def test_layer_norm_refusals():
    lib = C._lib.load()
    a = np.zeros(256, dtype=np.float32)
    p, odd = _ptr(a), ctypes.c_void_p(a.ctypes.data + 1)

    def fwd(dtype=F32, rows=2, width=8, x=p, ld=8, wt=F32, w=None, b=None, eps=1e-5, y=p, ldy=8, stats=None):
        return lib.cgtp_layer_norm_forward(dtype, rows, width, x, ld, wt, w, b, eps, y, ldy, stats, None)

    assert fwd(rows=0) == 0                       # nothing to do, nothing launched
    for bad in (dict(dtype=3), dict(rows=-1), dict(width=0), dict(x=None), dict(y=None), dict(ld=7), dict(ldy=7),
                dict(wt=BF16), dict(dtype=BF16, wt=F16), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(x=odd), dict(y=odd), dict(w=odd), dict(b=odd), dict(stats=odd)):
        assert fwd(**bad) == INVALID, bad
        assert lib.cgtp_last_error() != b""
    assert fwd(width=1 << 31) == UNSUPPORTED and fwd(rows=1 << 32, ld=8) == UNSUPPORTED

    ws = ctypes.c_size_t()
    assert lib.cgtp_layer_norm_backward_workspace_size(100, 8, ctypes.byref(ws)) == 0 and ws.value % 256 == 0
    assert lib.cgtp_layer_norm_backward_workspace_size(-1, 8, ctypes.byref(ws)) == INVALID
    assert lib.cgtp_layer_norm_backward_workspace_size(1, 8, None) == INVALID

    def bwd(rows=2, g=p, ldg=8, x=p, ld=8, stats=p, gx=p, ldgx=8, gw=None, gb=None, wsp=None, wsb=0):
        return lib.cgtp_layer_norm_backward(F32, rows, 8, g, ldg, x, ld, stats, F32, None, gx, ldgx, gw, gb, wsp, wsb,
                                            None)

    for bad in (dict(g=None), dict(stats=None), dict(ldg=7), dict(ldgx=7), dict(gw=odd, wsp=p, wsb=1 << 20),
                dict(gw=p, wsp=ctypes.c_void_p((a.ctypes.data + 511) // 256 * 256 + 4), wsb=1 << 20)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(rows=1000, gw=p) == WORKSPACE
    assert bwd(rows=1000, gb=p, wsp=ctypes.c_void_p((a.ctypes.data + 255) // 256 * 256), wsb=4) == WORKSPACE
    # a few rows need none
    assert lib.cgtp_layer_norm_backward_workspace_size(2, 8, ctypes.byref(ws)) == 0 and ws.value == 0


def test_irreps_norm_and_set_refusals():
    lib = C._lib.load()
    a = np.zeros(64, dtype=np.float32)
    assert lib.cgtp_irreps_norm_forward(None, F32, 1, _ptr(a), 8, F32, None, None, 1e-5, _ptr(a), 8, None, None) == INVALID
    assert lib.cgtp_norm_create(b"1x0e", None) == INVALID and lib.cgtp_params_create(None, None, 1, 0, None) == INVALID
    h = ctypes.c_void_p()
    assert lib.cgtp_params_create(None, None, 1, 0, ctypes.byref(h)) == INVALID
    assert lib.cgtp_params_create(None, None, 0, 8, ctypes.byref(h)) == INVALID
    # a set without a device is refused by every device call
    s = C.ParamSet([4], host_only=True)
    none = ctypes.c_void_p()
    assert lib.cgtp_adamw_step(s.handle, F32, none, F32, none, None, None, 1e-3, 0.9, 0.999, 1e-8, 1, None, None,
                               None) == INVALID
    assert b"HOST_ONLY" in lib.cgtp_last_error()
    assert lib.cgtp_grad_norm(s.handle, F32, none, None, 1.0, None, None, 0, None) == INVALID
    lib.cgtp_norm_destroy(None)
    lib.cgtp_params_destroy(None)


def test_norm_size_limits():
    # 2^29 values per irreps row, where the kernels' quotient e / (2l + 1) = e m >> 32 is exact
    for d in (3, 5, 7, 9, 11, 13):
        m = -(-2 ** 32 // d)
        assert all(e * m >> 32 == e // d for q in (1, 2 ** 28 // d, 2 ** 29 // d) for e in (q * d - 1, q * d))
        assert (2 ** 29 - 1) * (m * d - 2 ** 32) < 2 ** 32
    lib, h, ws = C._lib.load(), ctypes.c_void_p(), ctypes.c_size_t()
    assert lib.cgtp_norm_create(f"{2 ** 29 // 9 + 1}x4e".encode(), ctypes.byref(h)) == UNSUPPORTED and not h
    assert lib.cgtp_norm_create(f"{2 ** 28}x0e+{2 ** 28 + 1}x0o".encode(), ctypes.byref(h)) == UNSUPPORTED and not h
    assert lib.cgtp_norm_create(f"{2 ** 29 // 9}x4e".encode(), ctypes.byref(h)) == 0
    sizes = []
    for rows in (2 ** 31 - 1, 2 ** 31, 2 ** 63 - 1):   # more rows than a call takes: the largest call's
        assert lib.cgtp_irreps_norm_backward_workspace_size(h, rows, ctypes.byref(ws)) == 0
        sizes.append(ws.value)
    assert sizes[0] > 0 and len(set(sizes)) == 1
    lib.cgtp_norm_destroy(h)


def test_python_refuses_host_tensors():
    x = torch.zeros(3, 8)
    with pytest.raises(TypeError):
        C.layer_norm_forward(x)
    with pytest.raises(TypeError):
        C.layer_norm_forward(None)
    with pytest.raises(TypeError):
        C.layer_norm_backward(x, x, torch.zeros(2, 3))
    with pytest.raises(TypeError):
        C.irreps_norm_forward(C.NormPlan("8x0e"), x)
    s = C.ParamSet([24], host_only=True)
    with pytest.raises(TypeError):
        s.pointers([x])
    with pytest.raises(ValueError):
        s.pointers([x, x])
    with pytest.raises(ValueError):
        C.adamw_state(s, bits=16)


def test_import_without_device_support():
    # a torch built without devices has no raw stream: the package imports, host-only plans work
    code = """
import torch
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    del torch._C._cuda_getCurrentRawStream
import clebsch_gordan_tensor_node_amd as C
assert C.NormPlan("8x0e+2x1o").n_features == 14 and C.ParamSet([5], host_only=True).state_elems == 64
assert callable(C.train._raw_stream)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
