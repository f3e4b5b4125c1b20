"""CPU checks of the entry points of the operators for branching networks: every refusal
that happens on the host before a launch.  No device work is done here."""
import ctypes

import numpy as np
import pytest
import torch

C = pytest.importorskip("clebsch_gordan_tensor_node_amd")

INVALID, UNSUPPORTED, WORKSPACE = -1, -3, -5
F32, BF16, F16 = 0, 1, 2


def _ptr(a, by=0):
    return ctypes.c_void_p(a.ctypes.data + by)


@pytest.fixture(scope="module")
def lib():
    return C._lib.load()


def test_group_norm_refusals(lib):
    a = np.zeros(4096, dtype=np.float32)
    p, odd = _ptr(a), _ptr(a, 1)
    room = ctypes.c_void_p((a.ctypes.data + 255) // 256 * 256)

    def fwd(dtype=F32, rows=6, width=8, groups=2, samples=2, off=None, longest=0, x=p, ld=8, wt=F32, w=None, b=None, act=0, eps=1e-5,
            y=p, ldy=8, stats=None, ws=None, wsb=0):
        return lib.cgtp_group_norm_forward(dtype, rows, width, groups, samples, off, longest, x, ld, wt, w, b, act, eps, 0, y, ldy,
                                           stats, ws, wsb, None)

    def bwd(rows=6, width=8, groups=2, samples=2, off=None, g=p, ldg=8, x=p, ld=8, stats=p, wt=F32, w=None, b=None, act=0, gx=p, ldgx=8,
            gw=None, gb=None, ws=None, wsb=0, dtype=F32):
        return lib.cgtp_group_norm_backward(dtype, rows, width, groups, samples, off, 0, g, ldg, x, ld, stats, wt, w, b, act, gx, ldgx,
                                            gw, gb, ws, wsb, None)

    sizes = (dict(dtype=3), dict(rows=-1), dict(width=0), dict(groups=0), dict(groups=3), dict(groups=9), dict(samples=-1),
             dict(samples=4), dict(samples=0), dict(off=odd), dict(x=None), dict(ld=7), dict(wt=BF16), dict(dtype=BF16, wt=F16),
             dict(act=3), dict(act=-1), dict(x=odd), dict(w=odd), dict(b=odd))
    for bad in (*sizes, dict(longest=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(y=None), dict(ldy=7),
                dict(y=odd), dict(stats=odd)):
        assert fwd(**bad) == INVALID, bad
        assert lib.cgtp_last_error() != b""
    for bad in (*sizes, dict(g=None), dict(g=odd), dict(ldg=7), dict(stats=None), dict(stats=odd), dict(ldgx=7), dict(gx=odd),
                dict(gw=odd), dict(gb=odd)):
        assert bwd(**bad) == INVALID, bad
    for big in (dict(rows=1 << 31), dict(width=1 << 25, groups=1 << 25), dict(samples=1 << 31, off=p),
                dict(samples=1 << 30, off=p, width=1 << 10)):
        assert fwd(**big) == UNSUPPORTED and bwd(**big) == UNSUPPORTED, big
    assert fwd(rows=100000, samples=1) == WORKSPACE and bwd(rows=100000, samples=1) == WORKSPACE
    assert fwd(rows=100000, samples=1, ws=room, wsb=4) == WORKSPACE
    assert fwd(rows=100000, samples=1, ws=ctypes.c_void_p(room.value + 4), wsb=1 << 30) == INVALID
    assert bwd(gx=None) == 0   # nothing asked for, nothing launched


def test_group_norm_workspace(lib):
    ws = ctypes.c_size_t()

    def size(backward, dtype, rows, width, groups, samples, off, longest):
        assert lib.cgtp_group_norm_workspace_size(backward, dtype, rows, width, groups, samples, off, longest, ctypes.byref(ws)) == 0
        assert ws.value % 256 == 0
        return ws.value

    # a whole sample in a workgroup needs none; tiles do; the backward of several samples joins their sums
    some = ctypes.c_void_p(64)
    assert size(0, F32, 418, 64, 8, 1, None, 0) == 0 and size(1, F32, 418, 64, 8, 1, None, 0) == 0
    assert size(0, F32, 100000, 64, 8, 1, None, 0) > 0
    assert size(1, F32, 4000, 64, 8, 10, some, 400) >= 10 * 2 * 64 * 4
    assert size(0, BF16, 0, 64, 8, 0, some, 0) == 0
    assert lib.cgtp_group_norm_workspace_size(0, F32, 4, 8, 2, 1, None, 0, None) == INVALID
    assert lib.cgtp_group_norm_workspace_size(0, F32, 4, 8, 3, 1, None, 0, ctypes.byref(ws)) == INVALID


def test_route_refusals(lib):
    a = np.zeros(4096, dtype=np.float32)
    p, odd = _ptr(a), _ptr(a, 1)
    room = ctypes.c_void_p((a.ctypes.data + 255) // 256 * 256)

    def fwd(dtype=F32, rows=4, n=8, k=2, z=p, ld=8, ids=p, gates=p, counts=p, balance=p, slope=p, ws=room, wsb=4096):
        return lib.cgtp_route_forward(dtype, rows, n, k, z, ld, None, 0, 0, ids, gates, counts, balance, slope, ws, wsb, None)

    def bwd(dtype=F32, rows=4, n=8, k=2, z=p, ld=8, ids=p, slope=p, gg=p, gb=p, out=p, ldo=8):
        return lib.cgtp_route_backward(dtype, rows, n, k, z, ld, 0, 0, ids, slope, gg, gb, out, ldo, None)

    both = (dict(dtype=3), dict(rows=-1), dict(n=0), dict(k=0), dict(k=9), dict(z=None), dict(ld=7), dict(z=odd), dict(ids=None),
            dict(ids=odd), dict(slope=None), dict(slope=odd))
    for bad in (*both, dict(gates=None), dict(gates=odd), dict(counts=None), dict(counts=odd), dict(balance=None), dict(balance=odd),
                dict(ws=ctypes.c_void_p(room.value + 4))):
        assert fwd(**bad) == INVALID, bad
    for bad in (*both, dict(gg=odd), dict(gb=odd), dict(out=None), dict(out=odd), dict(ldo=7)):
        assert bwd(**bad) == INVALID, bad
    for big in (dict(rows=1 << 31), dict(n=1025, ld=1025), dict(n=100, k=65, ld=100)):
        assert fwd(**big) == UNSUPPORTED and bwd(**big) == UNSUPPORTED, big
    assert fwd(rows=100000, ws=None) == WORKSPACE and fwd(rows=100000, wsb=8) == WORKSPACE
    assert bwd(rows=0) == 0
    ws = ctypes.c_size_t()
    sizes = []
    for rows in (0, 1, 1024, 100000, 2 ** 31 - 1):
        assert lib.cgtp_route_workspace_size(rows, 8, ctypes.byref(ws)) == 0
        sizes.append(ws.value)
    assert sizes == sorted(sizes) and sizes[:3] == [0, 0, 0] and 0 < sizes[-1] < 1 << 20   # one workgroup needs none
    for rows, n in ((-1, 8), (4, 0)):
        assert lib.cgtp_route_workspace_size(rows, n, ctypes.byref(ws)) == INVALID
    assert lib.cgtp_route_workspace_size(4, 8, None) == INVALID
    assert lib.cgtp_route_workspace_size(4, 1025, ctypes.byref(ws)) == UNSUPPORTED


def test_gate_refusals(lib):
    a = np.zeros(64, dtype=np.float32)
    p, odd = _ptr(a), _ptr(a, 1)

    def bwd(edges=4, width=8, w=p, g=p, gate=p, out=p):
        return lib.cgtp_conv_gate_backward(edges, width, w, g, None, gate, out, None)

    for bad in (dict(edges=-1), dict(width=-1), dict(w=None), dict(g=None), dict(gate=None), dict(out=None), dict(w=odd), dict(g=odd),
                dict(gate=odd), dict(out=odd)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(edges=1 << 31) == UNSUPPORTED and bwd(width=1 << 31) == UNSUPPORTED
    assert bwd(edges=0) == 0


def test_python_refuses_host_tensors():
    x, e = torch.zeros(3, 8), torch.zeros(3)
    route = C.Route(torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2), torch.zeros(8, dtype=torch.int32), torch.zeros(1), torch.zeros(8),
                    False, False)
    for f in (lambda: C.group_norm_forward(x, 2), lambda: C.group_norm_forward(None, 2),
              lambda: C.group_norm_backward(x, x, torch.zeros(2, 1, 2), 2), lambda: C.route_forward(x, 2),
              lambda: C.route_backward(x, route), lambda: C.conv_gate_backward(x, x, e), lambda: C.conv_gate_backward(None, x, e)):
        with pytest.raises(TypeError):
            f()


def test_group_norm_workspace_of_what_is_asked_for(lib):
    ws = ctypes.c_size_t()

    def size(backward, rows, width, groups, samples, off, longest=0):
        assert lib.cgtp_group_norm_workspace_size(backward, F32, rows, width, groups, samples, off, longest, ctypes.byref(ws)) == 0
        return ws.value

    # the weights' gradients alone need a sum for each sample and column: not grad_x, nor one sample
    some = ctypes.c_void_p(64)
    assert size(1, 3000000, 8, 1, 3000000, None) == 3000000 * 2 * 8 * 4 and size(2, 3000000, 8, 1, 3000000, None) == 0
    for rows, samples in ((100000, 4), (4000, 10)):
        assert size(1, rows, 64, 8, samples, some) - size(2, rows, 64, 8, samples, some) in (samples * 2 * 64 * 4 + k for k in (-256, 0, 256))
    assert size(1, 100000, 64, 8, 1, None) == size(2, 100000, 64, 8, 1, None)
