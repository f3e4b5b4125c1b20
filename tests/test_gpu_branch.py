"""GPU checks of the operators for branching networks against their fp64 references.

Tolerances (u = 2^-24, the fp32 rounding unit).
Group norm.  Inputs: per channel a spread of 0.3 to 1.5 (clipped at 4 of it) around an offset of
  at most 2, |x| < 8, groups' spread above 0.3, weights in 0.1 to 1.9.  A thread sums at most
  some 40 differences x - K of size 2 (12 at most), its and the workgroups' joins add some 20
  roundings: the mean is off by 60 u 2 = 7e-6 at most, x - mean by as much, times rstd (below
  3) and the weight 5e-5.  The variance is off by some 3 (n + 20) u = 1e-5 of itself (see the
  kernel's comment; the mean of (K - mean)^2 over threads is the channel's own variance), rstd
  by half, h (below 8) by 4e-5, y by 8e-5.  fp32 is held to 2e-4 absolute; where rstd is larger
  (groups of few values), in proportion.
  grad_x: rstd times d w less the two means: d is off by |act''| < 1.2 times z's error, h as
  above, the means by some 100 u of terms of size 3 (|d h w|, 30 at most): 3 (2e-4 3 + 2e-5) =
  2e-3 at the most, typical errors being a hundredth: 1e-3 (times the scale squared).
  grad_weight, grad_bias: chains of at most 100 roundings in a row and z's and h's errors:
  (100 u + 1e-4) of the sum of the terms' magnitudes.
Routing.  exp to 3 u, a sum of n terms in a chain of 16 and a tree: p to 40 u of itself; balance
  and slope: p's sums, chains of some 500 at most before fp64: (500 + 40) u relative.
  grad_logits: p (u - sum(u p)): 100 u of p (|u| + sum |u| p), twice that if renormalised.
Gate: fp32 products and chains of W / 256 + 20: (W / 256 + 20) u of the sum of |w grad_w / gate|.
bf16 and fp16 outputs: the nearest value of the type to a number within these bounds.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle as O
import workloads as WL
from oracle import branch_oracle as B

C = pytest.importorskip("clebsch_gordan_tensor_node_amd")

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a device"
    return torch.device("cuda:0")


def _near(got, ref, tol, what):
    """got is within tol of ref, or in 16 bits the rounding of a number that is."""
    ref = np.asarray(ref)
    assert tuple(got.shape) == ref.shape, (what, got.shape, ref.shape)
    lo, hi = (torch.from_numpy(np.asarray(v)) for v in (ref - tol, ref + tol))
    if got.dtype != F32:
        lo, hi = lo.to(got.dtype).double(), hi.to(got.dtype).double()
    v = got.double().cpu()
    bad = ~(v.isfinite() & (lo <= v) & (v <= hi))
    assert not bad.any(), (what, int(bad.sum()), float((v - torch.from_numpy(ref)).abs().max()))


# ---- group norm ----------------------------------------------------------------------

def _rows(rng, n, f, dtype, dev, pad=0, first=0):
    """[n, f] rows inside rows `pad` wider, from column `first`, NaN beside them; in fp64."""
    v = rng.normal(size=(n, f)).clip(-4, 4) * rng.uniform(0.3, 1.5, size=f) + rng.uniform(-2, 2, size=f)
    wide = torch.full((n, f + pad), float("nan"), dtype=dtype, device=dev)
    t = wide[:, first:first + f]
    t.copy_(torch.from_numpy(v))
    return t, t.double().cpu().numpy()


def _weights(rng, n, dtype, dev):
    t = torch.from_numpy(1 + 0.3 * rng.normal(size=n).clip(-3, 3)).to(dtype).to(dev)
    return t, t.double().cpu().numpy()


def _bounds(rng, rows, samples, head=0, tail=0):
    """Ascending bounds of `samples` samples within rows [head, rows - tail)."""
    cuts = np.sort(rng.integers(head, max(rows - tail, head) + 1, size=max(samples - 1, 0)))
    return [head, *cuts.tolist(), max(rows - tail, head)]


def _offsets(cuts, dev):
    return torch.tensor(cuts, dtype=torch.int32, device=dev)


def _check(rows, width, groups, cuts, dev, dtype=F32, wdtype=F32, act="silu", longest=None, pad=0, first=0, seed=0,
           samples=None):
    rng = np.random.default_rng(seed)
    x, xr = _rows(rng, rows, width, dtype, dev, pad, first)
    (w, wr), (b, br) = _weights(rng, width, wdtype, dev), _weights(rng, width, wdtype, dev)
    samples = _offsets(cuts, dev) if samples is None else samples
    y, st = C.group_norm_forward(x, groups, w, b, samples=samples, activation=act, longest=longest)
    ry, rm, rr = B.group_norm_forward(xr, groups, cuts, wr, br, act)
    live = np.diff(cuts) > 0
    scale = max(1.0, np.abs(rr[live]).max(initial=0) / 3)
    _near(st[0], rm, 1e-5, "mean")
    _near(st[1], rr, 2e-5 * scale * rr, "rstd")
    _near(y, ry, 2e-4 * scale, "y")
    g, gr = _rows(rng, rows, width, dtype, dev, pad, 0)
    gx, gw, gb = C.group_norm_backward(g, x, st, groups, w, b, samples=samples, activation=act, longest=longest)
    rx, rw, rb = B.group_norm_backward(gr, xr, groups, cuts, wr, br, act)
    _near(gx, rx, 1e-3 * scale ** 2, "grad_x")
    aw, ab = np.zeros(width), np.zeros(width)
    for s, k, r, c in B._blocks(xr, cuts, groups):
        h = np.abs((xr[r, c] - rm[s, k]) * rr[s, k])
        aw[c] += (np.abs(gr[r, c]) * (h + 1) * 1.2).sum(axis=0)
        ab[c] += (np.abs(gr[r, c]) * 1.2).sum(axis=0)
    _near(gw, rw, (100 * U + 1e-4) * aw * scale, "grad_weight")
    _near(gb, rb, (100 * U + 1e-4) * ab * scale, "grad_bias")
    return x, g, w, b, samples, y, st, (gx, gw, gb)


WIDTHS = [(1, 1), (2, 1), (3, 3), (3, 1), (4, 2), (5, 1), (6, 2), (7, 7), (8, 8), (12, 4), (16, 2), (37, 1), (64, 8), (65, 5), (100, 25),
          (128, 4), (481, 13), (700, 7), (1024, 1), (1028, 1), (1312, 8), (2049, 3), (4100, 1), (5000, 2), (9001, 1)]


@pytest.mark.parametrize("whole", [True, False], ids=["whole", "tiles"])
@pytest.mark.parametrize("width,groups", WIDTHS)
def test_group_norm_widths(width, groups, whole, dev):
    # ragged samples with an empty one, as whole samples and (told of one as long as all rows) tiles
    rows = 3000 if width <= 128 else 700 if width <= 1312 else 150
    cuts = [0, rows // 3, rows // 3, rows // 3 + 33, rows]
    _check(rows, width, groups, cuts, dev, longest=None if whole else rows)


@pytest.mark.parametrize("dtype,wdtype", [(BF16, F32), (BF16, BF16), (F16, F32), (F16, F16)], ids=str)
@pytest.mark.parametrize("width,groups", [(1, 1), (3, 3), (7, 1), (8, 4), (16, 8), (64, 8), (128, 16), (130, 13), (481, 13), (1312, 8),
                                          (5000, 1)])
def test_group_norm_types(width, groups, dtype, wdtype, dev):
    rows = 900 if width <= 1312 else 200
    cuts = [0, 100, rows // 2, rows]
    _check(rows, width, groups, cuts, dev, dtype, wdtype, "gelu")
    _check(rows, width, groups, cuts, dev, dtype, wdtype, None, longest=rows, pad=5, first=3)


@pytest.mark.parametrize("rows", [1, 2, 5, 63, 418, 2600, 30011])
@pytest.mark.parametrize("width,groups", [(64, 8), (100, 4), (33, 3)])
def test_group_norm_row_counts(rows, width, groups, dev):
    for act in (None, "silu", "gelu"):
        _check(rows, width, groups, [0, rows], dev, act=act, samples=1)
    _check(rows, width, groups, [0, rows], dev, dtype=BF16, longest=rows)


@pytest.mark.parametrize("samples", [1, 2, 7, 300, 3000])
def test_group_norm_samples(samples, dev):
    # equal samples by their number, and ragged ones with rows outside them
    rows = 6000
    if rows % samples == 0:
        cuts = list(range(0, rows + 1, rows // samples))
        _check(rows, 24, 3, cuts, dev, samples=samples)
        _check(rows, 24, 3, cuts, dev, samples=samples, longest=rows)
    rng = np.random.default_rng(samples)
    # (groups of 16 values at least: few rows of 64 columns in 4 groups)
    for longest in (None, rows, 1):
        cuts = _bounds(rng, rows, samples, 13, 200)
        _check(rows, 64, 4, cuts, dev, longest=longest)
        _check(rows, 64, 4, cuts, dev, dtype=F16, longest=longest)


def test_group_norm_long_samples(dev):
    # one long sample, a few, and one that is far longer than told
    _check(100000, 40, 5, [0, 100000], dev)
    _check(60000, 128, 8, [100, 20000, 20001, 59000], dev, dtype=BF16, act="gelu")
    _check(20000, 64, 2, [0, 3, 19990, 20000], dev, longest=5)
    _check(20000, 64, 2, [0, 3, 19990, 20000], dev, dtype=BF16, longest=5)


def test_group_norm_row_samples(dev):
    # every row a sample: a layer norm of each group
    x, g, w, b, samples, y, st, grads = _check(500, 128, 2, list(range(501)), dev, samples=500, act=None)
    z, st2 = C.layer_norm_forward(x.reshape(1000, 64))
    assert (y - (z.view(500, 128) * w + b)).abs().max() < 2e-4
    assert (st.permute(0, 1, 2).reshape(2, 1000)[0] - st2[0]).abs().max() < 1e-5


def test_group_norm_rows_outside(dev):
    # NaN in rows that belong to no sample: 0 (or left as they were), gradient 0, nothing else changes
    for longest in (None, 1000):
        rng = np.random.default_rng(1)
        cuts = [50, 300, 300, 900]
        x, _ = _rows(rng, 1000, 36, F32, dev)
        g, _ = _rows(rng, 1000, 36, F32, dev)
        off = _offsets(cuts, dev)
        y, st = C.group_norm_forward(x, 4, samples=off, activation="silu", longest=longest)
        grads = C.group_norm_backward(g, x, st, 4, samples=off, activation="silu", longest=longest)
        for t in (x, g):
            t[:50], t[900:] = float("nan"), float("nan")
        y2, st2 = C.group_norm_forward(x, 4, samples=off, activation="silu", longest=longest)
        assert torch.equal(y2, y) and torch.equal(st2, st) and (y2[:50] == 0).all() and (y2[900:] == 0).all()
        again = C.group_norm_backward(g, x, st, 4, samples=off, activation="silu", longest=longest)
        assert all(torch.equal(a, c) for a, c in zip(grads, again)) and (again[0][900:] == 0).all()
        out = torch.full_like(x, 7.0)
        C.group_norm_forward(x, 4, samples=off, activation="silu", out=out, longest=longest)
        assert (out[:50] == 7).all() and (out[900:] == 7).all() and torch.equal(out[50:900], y[50:900])
    # no sample at all
    none = _offsets([3], dev)
    y, st = C.group_norm_forward(x, 4, samples=none)
    assert (y == 0).all() and st.shape == (2, 0, 4)
    gx, gw, gb = C.group_norm_backward(g, x, st, 4, samples=none)
    assert (gx == 0).all() and (gw == 0).all() and (gb == 0).all()


def test_group_norm_without_rows(dev):
    x = torch.empty(0, 12, device=dev)
    for samples, n in ((1, 1), (5, 5), (_offsets([0, 0, 0], dev), 2)):
        y, st = C.group_norm_forward(x, 3, samples=samples, eps=0.25)
        assert y.shape == (0, 12) and (st[0] == 0).all() and (st[1] == 2).all() and st.shape == (2, n, 3)
        gx, gw, gb = C.group_norm_backward(x, x, st, 3, samples=samples)
        assert gx.shape == (0, 12) and (gw == 0).all() and (gb == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_group_norm_constant_samples_are_their_bias(dtype, dev):
    # x - K is 0 throughout, so the mean is K, exactly, and y = act(bias)
    for longest in (None, 5000):
        for width, groups in ((12, 3), (37, 1), (128, 8), (1100, 1)):
            values = [100.0, 1000.0, -60000.0, 0.1, 8192.0]
            x = torch.tensor(values, device=dev).to(dtype).repeat_interleave(1000)[:, None].expand(5000, width).contiguous()
            b = torch.linspace(-1, 1, width, device=dev)
            y, st = C.group_norm_forward(x, groups, None, b, samples=5, longest=longest)
            assert torch.equal(y, b.to(dtype).expand(5000, width))
            assert torch.equal(st[0], x[::1000, :1].float().expand(5, groups))


def test_group_norm_infinities_stay_in_their_group(dev):
    for longest in (None, 600):
        rng = np.random.default_rng(2)
        x, _ = _rows(rng, 600, 16, F32, dev)
        off = _offsets([0, 200, 420, 600], dev)
        clean, st0 = C.group_norm_forward(x, 4, samples=off, activation="gelu", longest=longest)
        x[250, 5], x[599, 15] = float("inf"), float("nan")
        y, st = C.group_norm_forward(x, 4, samples=off, activation="gelu", longest=longest)
        hit = torch.zeros(600, 16, dtype=torch.bool, device=dev)
        hit[200:420, 4:8], hit[420:, 12:] = True, True
        assert y[hit].isnan().all() and torch.equal(y[~hit], clean[~hit])
        g, _ = _rows(rng, 600, 16, F32, dev)
        gx, _, _ = C.group_norm_backward(g, x, st, 4, samples=off, activation="gelu", longest=longest)
        assert gx[hit].isnan().all() and gx[~hit].isfinite().all()


def test_group_norm_large_arguments_of_the_activation(dev):
    # far from 0 the activations are 0 or z, with slope 0 or 1, also where exp overflows
    x = torch.tensor([[-1.0, 1.0]] * 8, device=dev)
    w = torch.full((2,), 1e4, device=dev)
    for act in ("silu", "gelu"):
        y, st = C.group_norm_forward(x, 1, w, activation=act, eps=0.0)
        assert (y[:, 0].abs() == 0).all() and (y[:, 1] - 1e4).abs().max() < 1e-2
        gx, gw, gb = C.group_norm_backward(torch.ones_like(x), x, st, 1, w, activation=act)
        assert gx.isfinite().all() and gb.tolist() == [0.0, 8.0]


@pytest.mark.parametrize("pad,first", [(1, 0), (1, 1), (7, 3)])
@pytest.mark.parametrize("width,groups", [(64, 4), (65, 5), (37, 1)])
def test_group_norm_strides(width, groups, pad, first, dev):
    for dtype in (F32, BF16):
        for longest in (None, 333):
            x, g, w, b, off, y, st, _ = _check(333, width, groups, [3, 100, 330], dev, dtype, pad=pad, first=first, longest=longest)
            wide = torch.full((333, width + pad), 7.0, dtype=dtype, device=dev)
            out, _ = C.group_norm_forward(x, groups, w, b, samples=off, activation="silu", longest=longest,
                                          out=wide[:, first:first + width])
            assert torch.equal(out[3:330], y[3:330])
            assert (wide[:, :first] == 7).all() and (wide[:, first + width:] == 7).all() and (out[:3] == 7).all()


@pytest.mark.parametrize("dtype", [F32, F16])
def test_group_norm_in_place(dtype, dev):
    for rows, width, groups, longest in ((700, 37, 1, None), (700, 37, 1, 700), (40000, 65, 5, None), (300, 2049, 3, 2),
                                         (5000, 66, 11, 3), (5, 3, 3, None)):
        rng = np.random.default_rng(3)
        x, _ = _rows(rng, rows, width, dtype, dev, 3, 1)
        off = _offsets([0, rows // 2, rows], dev)
        y, st = C.group_norm_forward(x, groups, samples=off, activation="silu", longest=longest)
        got, st2 = C.group_norm_forward(x, groups, samples=off, activation="silu", longest=longest, out=x)
        assert got.data_ptr() == x.data_ptr() and torch.equal(x, y) and torch.equal(st, st2)


def test_group_norm_optional_arguments(dev):
    for longest in (None, 500):
        rng = np.random.default_rng(4)
        x, xr = _rows(rng, 500, 30, F32, dev)
        g, gr = _rows(rng, 500, 30, F32, dev)
        cuts = [0, 200, 500]
        off = _offsets(cuts, dev)
        b, br = _weights(rng, 30, BF16, dev)
        y, st = C.group_norm_forward(x, 5, samples=off, longest=longest)
        _near(y, B.group_norm_forward(xr, 5, cuts)[0], 2e-4, "y")
        full = C.group_norm_backward(g, x, st, 5, samples=off, longest=longest)
        for got, ref in zip(full, B.group_norm_backward(gr, xr, 5, cuts)):
            _near(got, ref, 2e-3 if got.dim() == 2 else 5e-2, "gradient")
        for need in ((), ("x",), ("weight",), ("bias",), ("x", "bias"), ("weight", "bias")):
            some = C.group_norm_backward(g, x, st, 5, samples=off, need=need, longest=longest)
            for name, a, c in zip(("x", "weight", "bias"), some, full):
                assert (a is None) == (name not in need) and (a is None or torch.equal(a, c))
        xb = x.bfloat16()
        y, st = C.group_norm_forward(xb, 5, None, b, samples=off, activation="silu", longest=longest)
        ry = B.group_norm_forward(xb.double().cpu().numpy(), 5, cuts, None, br, "silu")[0]
        _near(y, ry, 2e-4, "y with a bias alone")
        assert C.group_norm_backward(g.bfloat16(), xb, st, 5, None, b, samples=off)[2].dtype == BF16


def test_group_norm_offsets_that_do_not_ascend(dev):
    # descending, negative, past the rows: no row outside x is touched
    room = torch.full((300, 20), 3.0, device=dev)
    x, keep = room[100:200], room.clone()
    for cuts in ([0, 5000, 10], [50, 20, 90, 10], [-7, 40, 2 ** 31 - 1], [2 ** 31 - 1, -2 ** 31, 7], [100, 0]):
        for longest in (None, 100):
            out = torch.full((300, 20), 5.0, device=dev)
            y, st = C.group_norm_forward(x, 4, samples=_offsets(cuts, dev), out=out[100:200], longest=longest)
            C.group_norm_backward(x, x, st, 4, samples=_offsets(cuts, dev), longest=longest)
            torch.cuda.synchronize()
            assert (out[:100] == 5).all() and (out[200:] == 5).all() and torch.equal(room, keep)


def test_group_norm_gradient_by_differences(dev):
    rng = np.random.default_rng(5)
    cuts = [0, 30, 100]
    for act in ("silu", "gelu"):
        x, xr = _rows(rng, 100, 12, F32, dev)
        g, gr = _rows(rng, 100, 12, F32, dev)
        (w, wr), (b, br) = _weights(rng, 12, F32, dev), _weights(rng, 12, F32, dev)
        off = _offsets(cuts, dev)
        _, st = C.group_norm_forward(x, 3, w, b, samples=off, activation=act)
        grads = [t.double().cpu().numpy() for t in C.group_norm_backward(g, x, st, 3, w, b, samples=off, activation=act)]
        loss = lambda x, w, b: (B.group_norm_forward(x, 3, cuts, w, b, act)[0] * gr).sum()  # noqa: E731
        h, args = 1e-5, (xr, wr, br)
        for k, got in enumerate(grads):
            d = rng.normal(size=got.shape)
            lo, hi = ([v + s * h * d if q == k else v for q, v in enumerate(args)] for s in (-1, 1))
            # up to 1200 gradients each within 1e-3 (typically 1e-5), and the differences' own error
            assert abs((got * d).sum() - (loss(*hi) - loss(*lo)) / (2 * h)) < 1e-3 + 1e-4 * abs((got * d).sum())


def test_group_norm_repeats_bitwise_on_another_stream(dev):
    rng = np.random.default_rng(6)
    for longest in (None, 9000):
        x, _ = _rows(rng, 9000, 96, F32, dev)
        g, _ = _rows(rng, 9000, 96, F32, dev)
        off = _offsets(_bounds(rng, 9000, 20), dev)

        def once():
            y, st = C.group_norm_forward(x, 6, samples=off, activation="silu", longest=longest)
            return (y, st, *C.group_norm_backward(g, x, st, 6, samples=off, activation="silu", longest=longest))

        first = once()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            again = once()
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, c) for a, c in zip(first, again))


def test_group_norm_places_past_32_bits(dev):
    # rows 2^21 elements apart: the last row's place is above 2^32 elements
    rows, ld, f = 2100, 1 << 21, 100
    rng = np.random.default_rng(7)
    buf = torch.empty(rows * ld, dtype=BF16, device=dev)
    x = buf.view(rows, ld)[:, :f]
    v, _ = _rows(rng, rows, f, BF16, dev)
    x.copy_(v)
    off = _offsets([0, 2000, 2100], dev)
    for longest in (None, rows):
        args = dict(samples=off, activation="silu", longest=longest)
        y, st = C.group_norm_forward(x, 4, **args)
        dense, st2 = C.group_norm_forward(v, 4, **args)
        assert torch.equal(y, dense) and torch.equal(st, st2)
        got, ref = C.group_norm_backward(x, x, st, 4, **args), C.group_norm_backward(v, v, st, 4, **args)
        assert all(torch.equal(a, c) for a, c in zip(got, ref))


def test_group_norm_in_a_graph(dev):
    # offsets change between replays: they are read on the device
    rng = np.random.default_rng(8)
    for longest in (None, 2000):
        x, _ = _rows(rng, 2000, 48, F32, dev)
        g, _ = _rows(rng, 2000, 48, F32, dev)
        off = _offsets([0, 500, 2000], dev)
        args = dict(samples=off, activation="silu", longest=longest)
        C.group_norm_backward(g, x, C.group_norm_forward(x, 6, **args)[1], 6, **args)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, st = C.group_norm_forward(x, 6, **args)
            grads = C.group_norm_backward(g, x, st, 6, **args)
        for cut in (500, 3, 1999, 0):
            x.copy_(_rows(rng, 2000, 48, F32, dev)[0])
            off.copy_(_offsets([0, cut, 1990], dev))
            graph.replay()
            torch.cuda.synchronize()
            want, st2 = C.group_norm_forward(x, 6, **args)
            assert torch.equal(y, want) and torch.equal(st, st2)
            assert all(torch.equal(a, c) for a, c in zip(grads, C.group_norm_backward(g, x, st2, 6, **args)))


# ---- routing -------------------------------------------------------------------------

def _logits(rng, rows, n, dtype, dev, ties=False, pad=0):
    v = rng.normal(size=(rows, n)) * 1.5 + rng.normal(size=n) * 0.5
    if ties:
        v = np.round(v)
    wide = torch.full((rows, n + pad), float("nan"), dtype=dtype, device=dev)
    t = wide[:, :n]
    t.copy_(torch.from_numpy(v))
    return t, t.double().cpu().numpy()


def _check_route(z, zr, k, dev, mask=None, renormalise=False, dense=False, seed=0):
    rows, n = zr.shape
    m = None if mask is None else mask.cpu().numpy()
    r = C.route_forward(z, k, mask=mask, renormalise=renormalise, dense=dense)
    ids, gates, counts, balance, slope = B.route_forward(zr, k, m, renormalise)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.array_equal(r.counts.cpu().numpy(), counts) and r.ids.dtype == r.counts.dtype == torch.int32
    want = B.dense_gates(ids, gates, n) if dense else gates
    _near(r.gates, want, 80 * U * want + 1e-38, "gates")
    _near(r.slope, slope, 2 * U * slope, "slope")
    _near(r.balance, [balance], 540 * U * abs(balance), "balance")
    rng = np.random.default_rng(seed)
    up = torch.from_numpy(rng.normal(size=want.shape)).float().to(dev)
    upr = up.double().cpu().numpy()
    if dense:   # the chosen entries
        upr = np.stack([upr[np.maximum(ids[:, i], 0), np.arange(rows)] for i in range(k)], axis=1)
    gb = torch.tensor([1.3], device=dev)
    p = B.softmax(zr)
    for a, b in ((up, gb), (up, None), (None, gb)):
        got = C.route_backward(z, r, a, b)
        ref = B.route_backward(zr, ids, slope, upr if a is not None else None, float(b) if b is not None else 0.0, renormalise)
        size = np.abs(upr).max(axis=1, initial=0)[:, None] + (1.3 * np.abs(slope)[None, :] + 1.3 * np.abs(slope).max(initial=0))
        share = np.maximum(p, B.dense_gates(ids, gates, n).T)   # a gate renormalised is above its p
        assert got.dtype == z.dtype
        _near(got, ref, 400 * U * share * size + 1e-37, "grad_logits")
    assert (C.route_backward(z, r) == 0).all()
    return r


@pytest.mark.parametrize("n,k", [(1, 1), (2, 1), (2, 2), (3, 2), (4, 4), (5, 3), (8, 2), (9, 9), (16, 4), (17, 3), (32, 8), (33, 5), (64, 6),
                                 (65, 1), (100, 16), (128, 8), (200, 64), (256, 8), (300, 7), (512, 64), (777, 10), (1024, 33)])
def test_route_sizes(n, k, dev):
    rng = np.random.default_rng(n)
    for dtype in (F32, BF16, F16):
        for dense, renormalise in ((False, False), (True, True)):
            z, zr = _logits(rng, 200, n, dtype, dev, ties=dense, pad=3 if dense else 0)
            mask = torch.from_numpy((rng.random(200) < 0.6).astype(np.uint8)).to(dev) if renormalise else None
            _check_route(z, zr, k, dev, mask, renormalise, dense)


@pytest.mark.parametrize("rows", [1, 2, 31, 255, 1024, 1025, 20011, 300000])
def test_route_rows(rows, dev):
    rng = np.random.default_rng(rows)
    for n, k in ((4, 1), (8, 2)) if rows > 100000 else ((4, 1), (8, 2), (60, 6), (256, 8)):
        z, zr = _logits(rng, rows, n, F32, dev)
        mask = torch.from_numpy((rng.random(rows) < 0.5).astype(np.uint8)).to(dev)
        _check_route(z, zr, k, dev, mask, rows % 2 == 0, n <= 8)


def test_route_ties_go_to_the_lowest_index(dev):
    for n in (6, 16, 40, 130, 700):
        z = torch.zeros(50, n, device=dev)
        z[::2] = -0.0
        z[:, n // 2] = 0.0
        r = C.route_forward(z, 5)
        assert (r.ids == torch.arange(5, device=dev, dtype=torch.int32)).all()
        z[:, n - 1] = 1.0
        r = C.route_forward(z, 5)
        assert (r.ids == torch.tensor([n - 1, 0, 1, 2, 3], device=dev, dtype=torch.int32)).all()


@pytest.mark.parametrize("n", [3, 8, 12, 40, 300])
def test_route_rows_that_are_masked_or_empty(n, dev):
    rng = np.random.default_rng(9)
    z, _ = _logits(rng, 400, n, F32, dev)
    z[5], z[6, 1:], z[7, :n - 1] = float("-inf"), float("-inf"), float("-inf")
    z[8] = torch.finfo(F32).min                      # the lowest finite value is a number
    z[9, 0] = torch.finfo(F32).min
    mask = torch.ones(400, dtype=torch.uint8, device=dev)
    mask[10:20] = 0
    z[12], z[13] = float("nan"), float("inf")        # masked: not looked at
    zr = z.double().cpu().numpy()
    clean = np.where(mask.cpu().numpy()[:, None] != 0, zr, 0.0)
    for dense in (False, True):
        r = C.route_forward(z, min(n, 3), mask, True, dense)
        ids, gates, counts, balance, slope = B.route_forward(clean, min(n, 3), mask.cpu().numpy(), True)
        assert np.array_equal(r.ids.cpu().numpy(), ids) and np.array_equal(r.counts.cpu().numpy(), counts)
        want = B.dense_gates(ids, gates, n) if dense else gates
        _near(r.gates, want, 80 * U * want + 1e-38, "gates")
        _near(r.balance, [balance], 540 * U * balance, "balance")
        up = torch.ones_like(r.gates)
        got = C.route_backward(z, r, up, torch.ones(1, device=dev))
        assert got.isfinite().all() and (got[5] == 0).all() and (got[10:20] == 0).all()
    # nothing left at all
    for none in (torch.zeros(400, dtype=torch.uint8, device=dev), None):
        zz = z if none is not None else torch.full_like(z, float("-inf"))
        r = C.route_forward(zz, 1, none, dense=True)
        assert (r.ids == -1).all() and (r.gates == 0).all() and (r.counts == 0).all() and r.balance.item() == 0 and (r.slope == 0).all()
        assert (C.route_backward(zz, r, torch.ones_like(r.gates), torch.ones(1, device=dev)) == 0).all()


def test_route_rows_that_are_not_finite(dev):
    rng = np.random.default_rng(10)
    for n in (5, 8, 70, 600):
        z, _ = _logits(rng, 300, n, F32, dev)
        ok = C.route_forward(z, 2)
        z[7, 3], z[9, 4] = float("nan"), float("inf")
        r = C.route_forward(z, 2)
        assert r.ids[7, 0] == 3 and r.ids[9, 0] == 4 and r.gates[7].isnan().all() and r.gates[9].isnan().all()
        keep = [i for i in range(300) if i not in (7, 9)]
        assert torch.equal(r.gates[keep], ok.gates[keep]) and torch.equal(r.ids[keep], ok.ids[keep]) and r.balance.isnan()
        assert (r.ids >= 0).all() and (r.ids < n).all() and r.counts.sum() == 600


def test_route_without_rows(dev):
    z = torch.empty(0, 6, device=dev)
    for dense in (False, True):
        r = C.route_forward(z, 2, dense=dense)
        assert (r.counts == 0).all() and r.balance.item() == 0 and r.ids.shape == (0, 2)
        assert C.route_backward(z, r, torch.empty_like(r.gates), r.balance).shape == (0, 6)


def test_route_backward_ignores_ids_out_of_range(dev):
    rng = np.random.default_rng(11)
    z, zr = _logits(rng, 50, 6, F32, dev)
    r = C.route_forward(z, 2)
    ids = r.ids.clone()
    ids[3, 1], ids[4, 0], ids[5, 1], ids[6, 0] = 6, -5, 2 ** 31 - 1, 1 << 20
    up = torch.ones(50, 2, device=dev)
    got = C.route_backward(z, r._replace(ids=ids), up)
    want = ids.cpu().numpy()
    want = np.where((want < 0) | (want >= 6), -1, want)
    _near(got, B.route_backward(zr, want, r.slope.cpu().numpy(), np.ones((50, 2))), 400 * U * 2, "grad_logits")


def test_route_repeats_bitwise_and_in_a_graph(dev):
    rng = np.random.default_rng(12)
    for n, k in ((8, 2), (100, 4)):
        z, _ = _logits(rng, 30000, n, F32, dev)
        up = torch.randn(n, 30000, device=dev)
        gb = torch.ones(1, device=dev)

        def once():
            r = C.route_forward(z, k, dense=True)
            return (*r[:5], C.route_backward(z, r, up, gb))

        first = once()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            again = once()
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, c) for a, c in zip(first, again))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = once()
        for _ in range(4):
            z.copy_(_logits(rng, 30000, n, F32, dev)[0])
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, c) for a, c in zip(held, once()))


# ---- gate ----------------------------------------------------------------------------

@pytest.mark.parametrize("width", [1, 3, 4, 40, 127, 128, 129, 255, 1023, 1024, 1312, 2176, 9001])
@pytest.mark.parametrize("edges", [1, 5, 700])
def test_gate_backward(edges, width, dev):
    rng = np.random.default_rng(width)
    w = torch.from_numpy(rng.normal(size=(edges, width))).float().to(dev)
    gate = torch.from_numpy(np.where(rng.random(edges) < 0.3, 0.0, 1 - rng.random(edges))).float().to(dev)
    mask = torch.from_numpy((rng.random(edges) < 0.8).astype(np.uint8)).to(dev)
    g = torch.from_numpy(rng.normal(size=(edges, width))).float().to(dev) * gate[:, None]
    for m in (None, mask):
        off = (gate == 0) | (False if m is None else m == 0)
        ww, gg = torch.where(off[:, None], float("nan"), w), torch.where(off[:, None], float("nan"), g)   # not read
        got = C.conv_gate_backward(ww, gg, gate, m)
        a = [t.double().cpu().numpy() for t in (w, g, gate)]
        ref = B.gate_backward(*a, None if m is None else m.cpu().numpy())
        size = B.gate_backward(np.abs(a[0]), np.abs(a[1]), a[2], None if m is None else m.cpu().numpy())
        _near(got, ref, (width / 256 + 20) * U * size, "grad_gate")
        out = torch.full((edges + 2,), 7.0, device=dev)
        assert C.conv_gate_backward(ww, gg, gate, m, out=out[1:-1]).data_ptr() == out[1:].data_ptr()
        assert torch.equal(out[1:-1], got) and out[0] == 7 and out[-1] == 7


def test_gate_backward_empty(dev):
    none = torch.empty(0, 8, device=dev)
    assert C.conv_gate_backward(none, none, none[:, 0].contiguous()).shape == (0,)
    narrow = torch.empty(4, 0, device=dev)
    assert (C.conv_gate_backward(narrow, narrow, torch.ones(4, device=dev)) == 0).all()


# ---- together ------------------------------------------------------------------------

def test_branches_together(dev):
    """Two branches of the 32-atom workload's convolution behind a routed, normalised hidden
    layer: forward and every gradient against the references run in the same order."""
    wl = WL.WORKLOADS["tiny"]
    pos, box, cell, rng = WL.positions(wl)
    rp, col, sh = O.neighbors(pos, box, wl.cutoff)
    ref = O.build_plan(wl.irreps_in, wl.irreps_sh, wl.l_out_max, wl.rule)
    plan = C.Plan(wl.irreps_in, wl.irreps_sh, wl.l_out_max, wl.rule)
    edges, n, k, hid, groups = len(col), 3, 2, 24, 4
    x, _, _ = WL.draw_payload(wl, rng, wl.n_atoms, ref.f_in, edges, ref.w_per_edge)
    rows, router = rng.normal(size=(edges, hid)).astype(np.float32), rng.normal(size=(hid, n)).astype(np.float32) / 3
    w = rng.normal(size=(n, edges, ref.w_per_edge)).astype(np.float32)
    gamma, beta = (1 + 0.2 * rng.normal(size=hid)).astype(np.float32), (0.2 * rng.normal(size=hid)).astype(np.float32)
    up = rng.normal(size=(n, wl.n_atoms, ref.f_out)).astype(np.float32)
    cuts = [0, edges // 3, edges]
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    graph = (to(pos), cell, to(rp.astype(np.int32)), to(col.astype(np.int32)), to(sh.astype(np.int8)))
    off, xt = _offsets(cuts, dev), to(x)

    hidden, st = C.group_norm_forward(to(rows), groups, to(gamma), to(beta), samples=off, activation="silu")
    logits = hidden @ to(router)
    r = C.route_forward(logits, k, renormalise=True, dense=True)
    outs = [C.conv_forward(plan, *graph, xt, to(w[b]), gate=r.gates[b]) for b in range(n)]
    grad_gates = torch.empty_like(r.gates)
    for b in range(n):
        _, gw, _ = C.conv_backward(plan, *graph, xt, to(w[b]), to(up[b]), gate=r.gates[b], need=("w",))
        C.conv_gate_backward(to(w[b]), gw, r.gates[b], out=grad_gates[b])
    gl = C.route_backward(logits, r, grad_gates, torch.full((1,), 0.5, device=dev))
    grads = C.group_norm_backward(gl @ to(router).t(), to(rows), st, groups, to(gamma), to(beta), samples=off, activation="silu")

    hr, _, _ = B.group_norm_forward(rows, groups, cuts, gamma, beta, "silu")
    zr = hr @ router.astype(np.float64)
    ids, gates, counts, balance, slope = B.route_forward(zr, k, None, True)
    gap = np.sort(zr, axis=1)
    assert (gap[:, n - k] - gap[:, n - k - 1]).min() > 1e-5   # no choice hangs on a rounding
    dense = B.dense_gates(ids, gates, n)
    assert np.array_equal(r.counts.cpu().numpy(), counts)
    gg = np.zeros_like(dense)
    for b in range(n):
        want = O.conv_forward(ref, pos, cell, rp, col, sh, x, w[b], gate=dense[b])
        assert np.linalg.norm(outs[b].double().cpu().numpy() - want) < 1e-5 * np.linalg.norm(want)
        gw = O.conv_backward(ref, pos, cell, rp, col, sh, x, w[b], up[b], gate=dense[b])[1]
        gg[b] = B.gate_backward(w[b], gw, dense[b])
    picked = np.stack([gg[ids[:, i], np.arange(edges)] for i in range(k)], axis=1)
    glr = B.route_backward(zr, ids, slope, picked, 0.5, True)
    want = B.group_norm_backward(glr @ router.T.astype(np.float64), rows, groups, cuts, gamma, beta, "silu")
    # gradients of order 10 to 100 through five operators of relative error 1e-6 to 1e-5 each
    for a, c in ((gl, glr), *zip(grads, want)):
        assert np.linalg.norm(a.double().cpu().numpy() - c) < 1e-4 * np.linalg.norm(c)


# ---- refusals ------------------------------------------------------------------------

def test_argument_checks(dev):
    x, st = torch.zeros(6, 8, device=dev), torch.zeros(2, 1, 2, device=dev)
    r = C.route_forward(x, 2)
    e = torch.zeros(6, device=dev)
    for f in (lambda: C.group_norm_forward(x.double(), 2), lambda: C.group_norm_forward(x.cpu(), 2),
              lambda: C.group_norm_forward(x, 2, torch.zeros(8, device=dev).half()),
              lambda: C.group_norm_forward(x, 2, torch.zeros(8)), lambda: C.group_norm_forward(x, 2, out=x.bfloat16()),
              lambda: C.group_norm_forward(x, 2, samples=torch.zeros(3, device=dev)),
              lambda: C.group_norm_forward(x, 2, samples=torch.zeros(3, dtype=torch.int64, device=dev)),
              lambda: C.group_norm_forward(x.bfloat16(), 2, torch.zeros(8, device=dev), torch.zeros(8, device=dev).bfloat16()),
              lambda: C.group_norm_backward(x.bfloat16(), x, st, 2), lambda: C.group_norm_backward(x, x, st.double(), 2),
              lambda: C.group_norm_backward(x, x, None, 2),
              lambda: C.route_forward(x.double(), 2), lambda: C.route_forward(x, 2, mask=torch.ones(6, device=dev)),
              lambda: C.route_backward(x, r, r.gates.double()), lambda: C.route_backward(x, r, None, torch.ones(2, device=dev)),
              lambda: C.route_backward(x, r._replace(ids=r.ids.long())),
              lambda: C.conv_gate_backward(x, x.double(), e), lambda: C.conv_gate_backward(x, x, None),
              lambda: C.conv_gate_backward(x, x, e, mask=e)):
        with pytest.raises(TypeError):
            f()
    for f in (lambda: C.group_norm_forward(x.view(2, 3, 8), 2), lambda: C.group_norm_forward(x.t(), 2),
              lambda: C.group_norm_forward(x[:1].expand(6, 8), 2), lambda: C.group_norm_forward(x, 2, activation="tanh"),
              lambda: C.group_norm_forward(x, 2, torch.zeros(7, device=dev)), lambda: C.group_norm_forward(x, 2, out=x[:3]),
              lambda: C.group_norm_forward(x, 2, samples=torch.zeros(0, dtype=torch.int32, device=dev)),
              lambda: C.group_norm_forward(x, 2, samples=torch.zeros(2, 2, dtype=torch.int32, device=dev)),
              lambda: C.group_norm_backward(x, x, st, 4), lambda: C.group_norm_backward(x[:2], x, st, 2),
              lambda: C.route_forward(x, 9), lambda: C.route_forward(x, 0), lambda: C.route_forward(x.t(), 2),
              lambda: C.route_forward(x, 2, mask=torch.ones(5, dtype=torch.uint8, device=dev)),
              lambda: C.route_backward(x[:, :7], r), lambda: C.route_backward(x[:3], r),
              lambda: C.route_backward(x, r, torch.zeros(8, 6, device=dev)), lambda: C.conv_gate_backward(x, x[:3], e),
              lambda: C.conv_gate_backward(x, x, e[:3]), lambda: C.conv_gate_backward(e, e, e),
              lambda: C.conv_gate_backward(x, x, e, out=e[:4])):
        with pytest.raises(ValueError):
            f()
    for f, code in ((lambda: C.group_norm_forward(x, 3), -1), (lambda: C.group_norm_forward(x, 0), -1),
                    (lambda: C.group_norm_forward(x, 2, samples=4), -1), (lambda: C.group_norm_forward(x, 2, samples=0), -1),
                    (lambda: C.group_norm_forward(x, 2, eps=-1.0), -1), (lambda: C.group_norm_forward(x, 2, longest=-1), -1),
                    (lambda: C.group_norm_forward(torch.zeros(100000, 8, device=dev), 2,
                                                  workspace=torch.empty(0, dtype=torch.uint8, device=dev)), -5),
                    (lambda: C.route_forward(torch.zeros(2, 1025, device=dev), 1), -3),
                    (lambda: C.route_forward(torch.zeros(2, 100, device=dev), 65), -3),
                    (lambda: C.route_forward(torch.zeros(100000, 8, device=dev), 2,
                                             workspace=torch.empty(0, dtype=torch.uint8, device=dev)), -5)):
        with pytest.raises(C.CgtpError) as err:
            f()
        assert err.value.code == code
    ws = ctypes.c_size_t()
    assert C._lib.load().cgtp_group_norm_workspace_size(0, 0, 6, 8, 2, 1, None, 0, ctypes.byref(ws)) == 0


def test_group_norm_of_small_values(dev):
    # without eps, x 2^-60 has the same y and gradients 2^60 times as large, bit for bit: every step
    # scales by a power of two, and nothing leaves fp32's normal range
    rng = np.random.default_rng(13)
    for longest in (None, 3000):
        x, _ = _rows(rng, 3000, 24, F32, dev)
        g, _ = _rows(rng, 3000, 24, F32, dev)
        args = dict(samples=_offsets([0, 1000, 3000], dev), activation="silu", longest=longest)
        y, st = C.group_norm_forward(x, 4, eps=0.0, **args)
        y2, st2 = C.group_norm_forward(x * 2.0 ** -60, 4, eps=0.0, **args)
        assert torch.equal(y, y2) and torch.equal(st[1] * 2.0 ** 60, st2[1])
        gx, gw, gb = C.group_norm_backward(g, x, st, 4, **args)
        gx2, gw2, gb2 = C.group_norm_backward(g, x * 2.0 ** -60, st2, 4, **args)
        assert torch.equal(gx * 2.0 ** 60, gx2) and torch.equal(gw, gw2) and torch.equal(gb, gb2)


# ---- sizes and uses at the ends of what the documents allow -----------------------------

def test_group_norm_without_eps_and_an_empty_sample(dev):
    # 1/sqrt(0) of a sample without rows reaches no gradient
    rng = np.random.default_rng(14)
    for longest in (None, 700):
        x, xr = _rows(rng, 700, 24, F32, dev)
        g, gr = _rows(rng, 700, 24, F32, dev)
        cuts = [0, 0, 300, 300, 700, 700]
        args = dict(samples=_offsets(cuts, dev), activation="silu", longest=longest)
        y, st = C.group_norm_forward(x, 3, eps=0.0, **args)
        assert y.isfinite().all() and (st[1, ::2] == float("inf")).all() and (st[0, ::2] == 0).all()
        full = C.group_norm_backward(g, x, st, 3, **args)
        ref = C.group_norm_backward(g, x, st[:, 1::2].contiguous(), 3, samples=_offsets([0, 300, 700], dev),
                                    activation="silu", longest=longest)
        for a, c in zip(full, ref):
            assert a.isfinite().all() and (a - c).abs().max() <= 1e-3 * (1 + c.abs().max())


@pytest.mark.parametrize("width,groups", [(1 << 20, 1), (1 << 20, 1 << 20), (1 << 20, 1 << 10), (1 << 24, 16)])
def test_group_norm_of_the_widest_rows(width, groups, dev):
    gen = torch.Generator(dev).manual_seed(15)
    x = torch.randn(9, width, device=dev, generator=gen)
    y, st = C.group_norm_forward(x, groups, samples=_offsets([0, 4, 9], dev), eps=1e-2)
    g = torch.randn(9, width, device=dev, generator=gen)
    gx, gw, gb = C.group_norm_backward(g, x, st, groups, samples=_offsets([0, 4, 9], dev))
    rw, rb = 0, 0
    for s, (i, j) in enumerate(((0, 4), (4, 9))):
        v, d = (t[i:j].double().view(j - i, groups, -1) for t in (x, g))
        mean = v.mean((0, 2), keepdim=True)
        rstd = ((v - mean).square().mean((0, 2), keepdim=True) + 1e-2).rsqrt()
        h = (v - mean) * rstd
        # as above, with rstd up to 10: h below 3 10 and its errors ten times
        assert (y[i:j] - h.view(j - i, -1)).abs().max() < 2e-3
        want = rstd * (d - d.mean((0, 2), keepdim=True) - h * (d * h).mean((0, 2), keepdim=True))
        assert (gx[i:j] - want.view(j - i, -1)).abs().max() < 2e-2
        rw, rb = rw + (d * h).sum(0).view(-1), rb + d.sum(0).view(-1)
    assert (gw - rw).abs().max() < 2e-2 and (gb - rb).abs().max() < 1e-4


def test_group_norm_of_millions_of_samples(dev):
    # one row each, in one group: a layer norm
    x = torch.randn(3000000, 8, device=dev, generator=torch.Generator(dev).manual_seed(16))
    y, st = C.group_norm_forward(x, 1, samples=3000000, eps=1e-2)
    z, st2 = C.layer_norm_forward(x, eps=1e-2)
    assert (y - z).abs().max() < 1e-4 and (st[0, :, 0] - st2[0]).abs().max() < 1e-5
    g = torch.randn(3000000, 8, device=dev, generator=torch.Generator(dev).manual_seed(17))
    gx, gw, _ = C.group_norm_backward(g, x, st, 1, samples=3000000)
    ref = C.layer_norm_backward(g, x, st2)
    assert (gx - ref[0]).abs().max() < 1e-2
    # 3e6 terms: both sums' chains stay below 3e6 / 1e4 + 100 additions
    assert (gw.double() - (g.double() * z.double()).sum(0)).abs().max() < 400 * U * 3e6


def test_group_norm_without_stats(dev):
    # the C entry point alone takes no stats; y is the same
    lib, stream = C._lib.load(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    rng = np.random.default_rng(18)
    for rows in (300, 60000):
        x, _ = _rows(rng, rows, 40, F32, dev)
        want, _ = C.group_norm_forward(x, 4, samples=1, activation="gelu")
        y, size = torch.empty_like(x), ctypes.c_size_t()
        assert lib.cgtp_group_norm_workspace_size(0, 0, rows, 40, 4, 1, None, 0, ctypes.byref(size)) == 0
        ws = torch.empty(max(size.value, 1), dtype=torch.uint8, device=dev)
        assert lib.cgtp_group_norm_forward(0, rows, 40, 4, 1, None, 0, x.data_ptr(), 40, 0, None, None, 2, 1e-5, 0, y.data_ptr(),
                                           40, None, ws.data_ptr(), size.value, stream) == 0
        assert torch.equal(y, want)


def test_calls_that_run_at_the_same_time(dev):
    # two streams, each with results and workspaces of its own, against the same calls alone
    rng = np.random.default_rng(19)
    sets = [(_rows(rng, 50000, 96, F32, dev)[0], _rows(rng, 50000, 96, F32, dev)[0]) for _ in range(2)]
    logits = [torch.from_numpy(rng.normal(size=(50000, n))).float().to(dev) for n in (8, 100)]

    def once(i):
        x, g = sets[i]
        y, st = C.group_norm_forward(x, 6, samples=5, activation="silu")
        r = C.route_forward(logits[i], 3, dense=True)
        return (y, st, *C.group_norm_backward(g, x, st, 6, samples=5, activation="silu"), *r[:5],
                C.route_backward(logits[i], r, r.gates, r.balance), C.conv_gate_backward(x, g, r.gates[0]))

    alone = [once(i) for i in range(2)]
    torch.cuda.synchronize()
    sides, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(4):
        for i, side in enumerate(sides):
            with torch.cuda.stream(side):
                got[i].append(once(i))
    torch.cuda.synchronize()
    for want, runs in zip(alone, got):
        for run in runs:
            assert all(torch.equal(a, c) for a, c in zip(want, run))


def test_route_of_many_rows(dev):
    # counts past 2^24 are whole; every workgroup takes many turns
    rows = 20000003
    logits = torch.zeros(rows, 2, dtype=BF16, device=dev)
    logits[-5:, 1] = 1
    r = C.route_forward(logits, 1)
    assert r.counts.tolist() == [rows - 5, 5] and (r.ids[:-5] == 0).all() and (r.ids[-5:] == 1).all()
    p = torch.softmax(logits.double(), 1).sum(0).cpu()
    balance = 2 * float((r.counts.cpu().double() * p).sum()) / rows ** 2
    # a thread's chain has rows / 2^18 = 77 additions, its workgroup's 8 steps
    assert abs(float(r.balance) - balance) < 200 * U * balance


def test_route_places_past_32_bits(dev):
    # logits' and dense gates' places above 2^32 bytes and 2^31 elements
    rows, n = 2200000, 1000
    logits = torch.zeros(rows, n, dtype=BF16, device=dev)
    logits[-3:, 997] = 30
    logits[-1, 3] = 29
    r = C.route_forward(logits, 2, dense=True)
    assert r.ids[-3:].tolist() == [[997, 0], [997, 0], [997, 3]] and (r.ids[:-3] == torch.tensor([0, 1], device=dev)).all()
    assert r.counts[[0, 1, 3, 997]].tolist() == [rows - 1, rows - 3, 1, 3]
    assert (r.gates[997, -3:] > 0.5).all() and (r.gates[997, :-3] == 0).all() and (r.gates[0, :-3] - 1e-3).abs().max() < 1e-8
    up = torch.zeros_like(r.gates)
    up[997, -1] = 1
    grad = C.route_backward(logits, r, up)
    p = torch.softmax(logits[-1].double(), 0)
    want = -p * p[997]
    want[997] += p[997]
    # 100 u of p (|u| + sum |u| p), twice, and the rounding to bf16
    assert ((grad[-1].double() - want).abs() <= 2.0 ** -8 * want.abs() + 400 * U).all()
    assert (grad[:-1] == 0).all()


def test_gate_backward_places_past_32_bits(dev):
    # rows of masked edges are not read, nor ever written here
    edges, width = 2300000, 1000
    w, g = (torch.empty(edges, width, device=dev) for _ in range(2))
    mask = torch.zeros(edges, dtype=torch.uint8, device=dev)
    gate = torch.full((edges,), 0.5, device=dev)
    for e in (0, 2147484, edges - 1):
        mask[e], w[e], g[e] = 1, 2.0, 3.0
    out = C.conv_gate_backward(w, g, gate, mask)
    assert out.nonzero().flatten().tolist() == [0, 2147484, edges - 1] and out[-1].item() == 12000.0


@pytest.mark.parametrize("width,groups", [(12, 3), (3, 1), (5000, 1)])
def test_group_norm_backward_without_rows_or_stats(width, groups, dev):
    # the C entry point alone takes no stats: without rows there are none to read
    lib, stream = C._lib.load(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    size = ctypes.c_size_t()
    for n in (1, 3, 3000):
        for off in (None, torch.zeros(n + 1, dtype=torch.int32, device=dev)):
            at = None if off is None else off.data_ptr()
            assert lib.cgtp_group_norm_workspace_size(1, 0, 0, width, groups, n, at, 0, ctypes.byref(size)) == 0
            ws = torch.empty(max(size.value, 1), dtype=torch.uint8, device=dev)
            grads = torch.full((2, width), 7.0, device=dev)
            assert lib.cgtp_group_norm_backward(0, 0, width, groups, n, at, 0, None, width, None, width, None, 0, None, None, 1, None,
                                                width, grads[0].data_ptr(), grads[1].data_ptr(), ws.data_ptr(), size.value, stream) == 0
            assert (grads == 0).all()


@pytest.mark.parametrize("rows,width,groups,dtype,longest,lead", [
    (60000, 1024, 1, F32, 1, 8), (200000, 64, 4, F32, 1, 400), (60000, 1024, 1, BF16, 1, 40), (300000, 1024, 2, F32, None, 8),
    (400000, 1024, 1, BF16, None, 8)], ids=str)
def test_group_norm_threads_of_many_rows(rows, width, groups, dtype, longest, lead, dev):
    """Samples far longer than told, and tiles of more than 64 rows a thread, with first rows 100
    deviations off: threads' first values, about which they sum.

    A thread's sums are chains of 64 additions, closed about the mean so far, then of n / 64.  Of
    |x - K| < 110: the first run's sum is below 7000, off by 64 u 7000 = 0.03, the later ones' by less
    (K nears the mean as 1 / runs: 0.2 in all), the mean by 0.2 / 3000 at the most, 2e-5 where n =
    60000.  Squares: a run's are below 8e5, off by 64 u 8e5 = 3, the moves of K by as much, in all
    some 10 of the n + 1e4 (lead / slices) that they sum to: 1e-3 for n = 3000 + 6e4 / 64 at the
    worst, where 64 threads' errors of both signs are joined; 1e-4 + n u / 64 otherwise.  rstd is off
    by half of that.  grad_bias of equal terms: (64 + n / 64 + 30) u of their sum."""
    gen = torch.Generator(dev).manual_seed(21)
    x = torch.randn(rows, width, device=dev, generator=gen)
    x[:lead] += 100
    x = x.to(dtype)
    y, st = C.group_norm_forward(x, groups, samples=1, longest=longest)
    v = x.double().view(rows, groups, -1)
    mean = v.mean((0, 2), keepdim=True)
    var = (v - mean).square().mean((0, 2), keepdim=True)
    rstd = (var + 1e-5).rsqrt()
    assert (st[0, 0] - mean.flatten()).abs().max() < 3e-5
    assert (st[1, 0] / rstd.flatten() - 1).abs().max() < 2e-4
    # the rounding of y, of at most some 100, and rstd's error of it
    h = ((v - mean) * rstd).view(rows, width)
    assert ((y.double() - h).abs() <= (torch.finfo(dtype).eps / 2 + 2e-4) * h.abs() + 5e-5).all()
    del v
    # the same bounds for the sums of the backward: all of one sign, and equal
    g = torch.full_like(x, 0.1)
    gx, gw, gb = C.group_norm_backward(g, x, st, groups, samples=1, longest=longest)
    d = float(g[0, 0])
    assert (gb.double() / (d * rows) - 1).abs().max() < (64 + rows / 64 + 30) * U
    # h within 2e-4 of itself and 5e-5, and the chains, of sum |d h|
    assert ((gw.double() - d * h.sum(0)).abs() <= d * ((2e-4 + (94 + rows / 64) * U) * h.abs().sum(0) + 5e-5 * rows)).all()
    # d - mean(d) - h mean(d h) = -h mean(d h), and mean(d h) is 0 but for its error
    assert (gx.double().abs() <= rstd.max() * d * (1 + rows / 64) * 2 * U + (h.abs() + 1) * d * 3e-4).all()


@pytest.mark.parametrize("n", [6, 16, 20, 64, 100, 200, 400, 1000])
def test_route_backward_of_a_branch_twice_in_a_row(n, dev):
    # ids that no forward writes: the gates' gradients of one branch are added in the choices' order,
    # which shows in 2^24 + 1 - 2^24 (0, and 1 in another order)
    z = torch.randn(300, n, device=dev, generator=torch.Generator(dev).manual_seed(22))
    r = C.route_forward(z, 6)
    ids = torch.tensor([n - 1, 2, n - 1, 2, n - 1, 2], dtype=torch.int32, device=dev).repeat(300, 1)
    ids[::3] = r.ids[::3]   # among rows as the forward leaves them
    up = torch.randn(300, 6, device=dev, generator=torch.Generator(dev).manual_seed(23))
    big = 2.0 ** 24
    up[1::3] = torch.tensor([big, 1, 1, big, -big, -big], device=dev)
    total = up.clone()
    for i in (2, 4):
        total[:, 0] += up[:, i]   # in fp32, in order
        total[:, 1] += up[:, i + 1]
    once = torch.stack([torch.where(torch.arange(300, device=dev) % 3 == 0, r.ids[:, i], i and 2 if i else n - 1) for i in range(2)], 1).int()
    for dense in (False, True):
        if dense:   # one gradient for a branch and row, added as often as it is there
            u = torch.randn(n, 300, device=dev, generator=torch.Generator(dev).manual_seed(24))
            got = C.route_backward(z, r._replace(ids=ids, dense=True), u)
            at = ids.long()
            flat = torch.gather(u.t(), 1, at)
            want_up = torch.stack([flat[:, 0] + flat[:, 2] + flat[:, 4], flat[:, 1] + flat[:, 3] + flat[:, 5]], 1)
        else:
            got = C.route_backward(z, r._replace(ids=ids), up)
            want_up = total[:, :2]
        want = C.route_backward(z, r._replace(ids=once.contiguous()), want_up.contiguous())
        rows = torch.arange(300, device=dev) % 3 != 0
        assert torch.equal(got[rows], want[rows])
        as_forward = C.route_backward(z, r._replace(dense=dense), u if dense else up)
        assert torch.equal(got[~rows], as_forward[~rows])


@pytest.mark.parametrize("groups", [1, 4096])
def test_group_norm_gelu_in_32_bits(groups, dev):
    """z of two rows, 1 and -1 times the weight: mean 0 and rstd 1 exactly, so that z is exact.
    q = 1 - cdf(|z|): exp's roundings 4 u and z^2 / 2 u of its argument, the reciprocal's 2 u twice,
    the polynomial's (partial sums below 1) 2 u, its fit 0.5 u, products 2 u: (13 + z^2 / 2) u of q
    itself, one more for y; the rounding of 1 - q where z > 0."""
    n = 1 << 16
    gen = torch.Generator(dev).manual_seed(25)
    z = torch.cat([torch.randn(n // 2, device=dev, generator=gen), 16 * torch.rand(n // 2, device=dev, generator=gen) - 8])
    x = torch.ones(2, n, device=dev)
    x[1] = -1
    y, st = C.group_norm_forward(x, groups, z, activation="gelu", eps=0.0)
    assert (st[0] == 0).all() and (st[1] == 1).all()
    zz = torch.stack([z, -z]).double()
    q = torch.special.erfc(zz.abs() * 0.5 ** 0.5) / 2
    cdf = torch.where(zz < 0, q, 1 - q)
    off = (14 + zz.square() / 2) * U * q + (zz > 0) * 2 * U
    assert ((y.double() - zz * cdf).abs() <= zz.abs() * off + 1e-37).all()
    g = torch.tensor([[1.0], [0.0]], device=dev).expand(2, n).contiguous()
    grad_bias = C.group_norm_backward(g, x, st, groups, z, activation="gelu")[2].double()
    density = torch.exp(-zz[0].square() / 2) * (2 * torch.pi) ** -0.5
    # the slope cdf + z density: the density's 4 u and z^2 / 2 u, and a product's and a sum's rounding
    tol = off[0] + zz[0].abs() * density * (6 + zz[0].square() / 2) * U + 2 * U * (cdf[0] + zz[0] * density).abs() + 1e-37
    assert ((grad_bias - (cdf[0] + zz[0] * density)).abs() <= tol).all()


def test_group_norm_backward_of_x_alone_needs_less_room(dev):
    lib, stream = C._lib.load(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    rng = np.random.default_rng(26)
    for rows, width, groups, samples, longest in ((30000, 8, 1, 30000, 0), (9000, 64, 4, 30, 0), (9000, 64, 4, 30, 9000), (60000, 64, 4, 1, 0)):
        x, _ = _rows(rng, rows, width, F32, dev)
        g, _ = _rows(rng, rows, width, F32, dev)
        args = dict(samples=samples, activation="silu", longest=longest)
        _, st = C.group_norm_forward(x, groups, eps=1e-2, **args)
        want = C.group_norm_backward(g, x, st, groups, **args)[0]
        size = ctypes.c_size_t()
        assert lib.cgtp_group_norm_workspace_size(2, 0, rows, width, groups, samples, None, longest, ctypes.byref(size)) == 0
        room = torch.full((size.value + 512,), 77, dtype=torch.uint8, device=dev)
        gx = torch.empty_like(x)
        at = room.data_ptr() if size.value else None
        assert lib.cgtp_group_norm_backward(0, rows, width, groups, samples, None, longest, g.data_ptr(), width, x.data_ptr(), width,
                                            st.data_ptr(), 0, None, None, 1, gx.data_ptr(), width, None, None, at, size.value, stream) == 0
        assert torch.equal(gx, want) and (room[size.value:] == 77).all()
        assert torch.equal(C.group_norm_backward(g, x, st, groups, need=("x",), **args)[0], want)
