"""GPU checks of the training operators against their fp64 references.

Tolerances (u = 2^-24, the fp32 rounding unit).  Inputs are rows of spread 0.5 to 1.5
around an offset of at most 4, |x| < 10, and weights below 2.
  forward: x - mu carries the mean's error, some 10 u of |x| (partial sums of a thread and
    a tree), and its own rounding; rstd (at most 1/0.4) some 30 u: 10 * 10 u * 2.5 + 30 u * 6
    below 3e-5 for |h| < 6; times the weight.  fp32 is held to 5e-5 absolute.
  grad_x: the same terms with two sums more: 1e-4 absolute, |grad_x| being of order 1 to 10.
  grad_weight, grad_bias: partial sums of at most 100 terms in a chain and a tree: 100 u of
    the sum of the terms' magnitudes, and h's error (3e-5 / 6 relative at most) of it.
  bf16 and fp16 outputs: the nearest value of the type to a number within these bounds.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import train_oracle as T

C = pytest.importorskip("clebsch_gordan_tensor_node_amd")

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SPECS = [1, 2, 3, 4, 5, 8, 16, 17, 63, 64, 65, 128, 129, 257, 480, 512, 513, 1024, 1025, 1312, 2048, 2049, 4096, 4097, 8192,
         8193, 16384, 16385, 40001, "16x0e+8x1e+16x1o", "1x0e", "1x0o+1x1o+1x6e", "128x0e+64x1o+32x2e+32x3o",
         "640x0e+1024x1o+1280x2e", "5x0e+3x0o+7x4e+2x0e", "+".join(["3x0e+1x1o"] * 32), "20000x0e+3x1o+7000x1o+600x0e",
         "1152x4e+9x0e+2000x0o"]


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a device"
    return torch.device("cuda:0")


def _rows(rng, n, f, dtype, dev, pad=0, first=0):
    """[n, f] rows inside rows `pad` wider, from column `first`; and their values in fp64."""
    v = rng.normal(size=(n, f)).clip(-4, 4) * rng.uniform(0.5, 1.5, size=(n, 1)) + rng.uniform(-3, 3, size=(n, 1))
    wide = torch.full((n, f + pad), float("nan"), dtype=dtype, device=dev)
    t = wide[:, first:first + f]
    t.copy_(torch.from_numpy(v))
    return t, t.double().cpu().numpy()


def _weights(rng, n, dtype, dev):
    t = torch.from_numpy(1 + 0.3 * rng.normal(size=n).clip(-3, 3)).to(dtype).to(dev)
    return t, t.double().cpu().numpy()


def _call(spec, x, w, b, eps=1e-5, **kw):
    if isinstance(spec, int):
        y, st = C.layer_norm_forward(x, w, b, eps, **kw)
        return y, st.view(2, x.shape[0], 1)
    return C.irreps_norm_forward(C.NormPlan(spec), x, w, b, eps, **kw)


def _grads(spec, g, x, st, w, **kw):
    if isinstance(spec, int):
        return C.layer_norm_backward(g, x, st.view(2, x.shape[0]), w, **kw)
    return C.irreps_norm_backward(C.NormPlan(spec), g, x, st, w, **kw)


def _shape(spec):
    t = T.row_terms(spec) if isinstance(spec, int) else T.norm_terms(spec)
    return (t, sum(m * d for _, m, d, _, _ in t), sum(m for _, m, _, _, _ in t),
            sum(m for _, m, _, _, b in t if b is not None))


def _near(got, ref, tol, what):
    """got is within tol of ref, or in 16 bits the rounding of a number that is."""
    assert tuple(got.shape) == ref.shape, (what, got.shape, ref.shape)
    lo, hi = (torch.from_numpy(np.asarray(v)) for v in (ref - tol, ref + tol))
    if got.dtype != torch.float32:
        lo, hi = lo.to(got.dtype).double(), hi.to(got.dtype).double()
    v = got.double().cpu()
    assert v.isfinite().all() and ((lo <= v) & (v <= hi)).all(), (what, float((v - torch.from_numpy(ref)).abs().max()))


def _check(spec, rows, dtype, wdtype, dev, pad=0, first=0, seed=0):
    rng = np.random.default_rng(seed)
    terms, f, nw, nb = _shape(spec)
    x, xr = _rows(rng, rows, f, dtype, dev, pad, first)
    (w, wr), (b, br) = _weights(rng, nw, wdtype, dev), _weights(rng, nb, wdtype, dev)
    y, st = _call(spec, x, w, b)
    ry, rm, rr = T.norm_forward(xr, terms, wr, br)
    scale = max(1.0, np.abs(rr).max(initial=0) / 2.5)   # a row of one or two values may have a large rstd
    _near(y, ry, 5e-5 * scale, "y")
    _near(st[0], rm, 100 * U, "mean")
    _near(st[1], rr, (60 * U + 2e-5 * scale) * rr, "rstd")
    g, gr = _rows(rng, rows, f, dtype, dev, pad, 0)
    gx, gw, gb = _grads(spec, g, x, st, w)
    rx, rw, rb = T.norm_backward(gr, xr, terms, wr)
    _near(gx, rx, 1e-4 * scale ** 2, "grad_x")
    aw, ab = np.zeros(nw), np.zeros(nb)
    for k, (off, m, d, w0, b0) in enumerate(terms):
        q = np.abs(gr[:, off:off + m * d]).reshape(rows, m, d)
        h = np.abs((xr[:, off:off + m * d].reshape(rows, m, d) - rm[:, k, None, None]) * rr[:, k, None, None])
        aw[w0:w0 + m] = (q * (h + 1)).sum(axis=(0, 2))
        if b0 is not None:
            ab[b0:b0 + m] = q.sum(axis=(0, 2))
    _near(gw, rw, (100 * U + 2e-5) * aw * scale, "grad_weight")
    _near(gb, rb, 100 * U * ab, "grad_bias")
    return x, g, w, b, y, st, (gx, gw, gb)


@pytest.mark.parametrize("spec", SPECS, ids=lambda s: str(s)[:30])
def test_norm_widths(spec, dev):
    _check(spec, 7, torch.float32, torch.float32, dev)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("spec", [1, 5, 7, 8, 33, 64, 129, 257, 513, 1025, 1312, 2049, 4097, 8193, 16384, 20000,
                                  "128x0e+64x1o+32x2e+32x3o", "5x0e+3x0o+7x4e+2x0e", "18000x0e+3x1o+300x2e"], ids=str)
def test_norm_types(spec, dtype, dev):
    _check(spec, 9, dtype, torch.float32, dev)
    _check(spec, 9, dtype, dtype, dev, pad=3, first=1)


@pytest.mark.parametrize("rows", [1, 2, 31, 257, 4000])
@pytest.mark.parametrize("spec", [3, 7, 16, 30, 77, 128, 480, 1030, "16x0e+8x1e+16x1o"], ids=str)
def test_norm_row_counts(spec, rows, dev):
    # one workgroup per term, and many with their partial sums
    _check(spec, rows, torch.float32, torch.float32, dev)
    if rows > 31:
        _check(spec, rows, torch.bfloat16, torch.float32, dev)


@pytest.mark.parametrize("spec,rows", [(1312, 60000), ("128x0e+64x1o+32x2e+32x3o", 100000)], ids=str)
def test_norm_rows_that_outgrow_the_cache(spec, rows, dev):
    # more than 256 MB: every row is what it is in a call of its own size, bit for bit, and the
    # weight's gradient is the sum of the parts'
    terms, f, nw, nb = _shape(spec)
    gen = torch.Generator(device=dev).manual_seed(0)
    x, g = (torch.randn(rows, f, device=dev, generator=gen) for _ in range(2))
    w, b = torch.randn(nw, device=dev, generator=gen), torch.randn(nb, device=dev, generator=gen)
    y, st = _call(spec, x, w, b)
    gx, gw, gb = _grads(spec, g, x, st, w)
    sw, sb = torch.zeros(nw, dtype=torch.float64, device=dev), torch.zeros(nb, dtype=torch.float64, device=dev)
    for r in range(0, rows, 5000):
        yr, sr = _call(spec, x[r:r + 5000], w, b)
        assert torch.equal(y[r:r + 5000], yr)
        gxr, gwr, gbr = _grads(spec, g[r:r + 5000], x[r:r + 5000], sr, w)
        assert torch.equal(gx[r:r + 5000], gxr)
        sw += gwr
        sb += gbr
    # sums of `rows` terms of size below 25 |g| |h| in 5000-row and in longer chains: 100 u of
    # the sum of magnitudes, which is below 13 rows for the widest channel
    bound = 100 * U * 13 * rows
    assert (gw - sw).abs().max() < bound and (gb - sb).abs().max() < bound


def _small_integers(shape, dtype, dev, gen):
    return torch.randint(-3, 4, shape, device=dev, generator=gen).to(dtype)


@pytest.mark.parametrize("spec", [33, 700, 1000, 3000, 5000, 12000, "128x0e+64x1o+32x2e+32x3o"], ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_norm_past_the_cache_in_every_type(dtype, spec, dev):
    # calls that move more than 256 MB, forward and backward: rows bit for bit as in smaller
    # calls; of small integers with mean 0 and rstd 1 (h = x) the sums of the weight's and bias's
    # gradients are whole numbers below 2^24, so that a row too few or too many shows
    terms, f, nw, nb = _shape(spec)
    rows = (1 << 28) // (2 * f * torch.finfo(dtype).bits // 8) + 77
    gen = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn(rows, f, device=dev, generator=gen).to(dtype)
    w, b = torch.randn(nw, device=dev, generator=gen), torch.randn(nb, device=dev, generator=gen)
    y, st = _call(spec, x, w, b)
    part = (rows + 3) // 4
    for r in range(0, rows, part):
        yr, sr = _call(spec, x[r:r + part], w, b)
        assert torch.equal(y[r:r + part], yr) and torch.equal(st[:, r:r + part], sr)
    del y
    x, g = _small_integers((rows, f), dtype, dev, gen), _small_integers((rows, f), dtype, dev, gen)
    st = torch.stack([torch.zeros(rows, len(terms), device=dev), torch.ones(rows, len(terms), device=dev)])
    gx, gw, gb = _grads(spec, g, x, st, w)
    for r in range(0, rows, part):
        gxr, _, _ = _grads(spec, g[r:r + part], x[r:r + part], st[:, r:r + part].contiguous(), w)
        assert torch.equal(gx[r:r + part], gxr)
    _check_whole_sums(terms, g, x, gw, gb)


def _check_whole_sums(terms, g, x, gw, gb):
    for off, m, d, w0, b0 in terms:
        q, h = g[:, off:off + m * d].float(), x[:, off:off + m * d].float()
        want = (q * h).sum(0, dtype=torch.float64).view(m, d).sum(1)
        assert torch.equal(gw[w0:w0 + m].double(), want)
        if b0 is not None:
            assert torch.equal(gb[b0:b0 + m].double(), q.sum(0, dtype=torch.float64))


@pytest.mark.parametrize("spec", ["5x0e+3x0o+7x4e+2x0e+9x1o+33x0e+8x2e+1x0o+64x0e", "+".join(["3x0e+1x1o"] * 32), 600, 1000, 1024,
                                  "1x0e+700x0e+100x1o"], ids=lambda s: str(s)[:30])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_partial_sums_of_many_rows(dtype, spec, dev):
    # more than 8 terms, and 16 elements a lane: several workgroups per term and the second launch
    _check(spec, 4000, dtype, torch.float32, dev)
    terms, f, nw, nb = _shape(spec)
    gen = torch.Generator(device=dev).manual_seed(2)
    for rows in (200, 9001):
        x, g = _small_integers((rows, f), dtype, dev, gen), _small_integers((rows, f), dtype, dev, gen)
        st = torch.stack([torch.zeros(rows, len(terms), device=dev), torch.ones(rows, len(terms), device=dev)])
        _, gw, gb = _grads(spec, g, x, st, torch.ones(nw, device=dev))
        _check_whole_sums(terms, g, x, gw, gb)


@pytest.mark.parametrize("pad,first", [(1, 0), (1, 1), (7, 3), (64, 32)])
@pytest.mark.parametrize("spec", [64, 65, 1312, "128x0e+64x1o+32x2e+32x3o"], ids=str)
def test_norm_strides(spec, pad, first, dev):
    # rows inside wider ones, starting anywhere: what lies beside them (NaN) is not read into
    # the result and the output's neighbours are not written
    for dtype in (torch.float32, torch.bfloat16):
        x, g, w, b, y, st, _ = _check(spec, 33, dtype, torch.float32, dev, pad, first)
        f = x.shape[1]
        wide = torch.full((33, f + pad), 7.0, dtype=dtype, device=dev)
        out, _ = _call(spec, x, w, b, out=wide[:, first:first + f])
        assert torch.equal(out, y)
        assert (wide[:, :first] == 7).all() and (wide[:, first + f:] == 7).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("spec,rows", [(3, 500), (7, 500), (100, 500), (481, 300), (700, 300), (1312, 300), (2049, 100), (5000, 50),
                                       (12001, 40), (16384, 40), (30001, 40), ("5x0e+3x0o+7x4e+2x0e", 500), (700, 140000),
                                       ("20000x0e+3x1o+7000x1o+600x0e", 30), ("128x0e+64x1o+32x2e+32x3o", 70000)], ids=str)
def test_norm_in_place(spec, rows, dtype, dev):
    # y in x's place, in every layout, within and past the cache: bit for bit what it is elsewhere
    terms, f, nw, nb = _shape(spec)
    gen = torch.Generator(device=dev).manual_seed(4)
    wide = torch.randn(rows, f + 3, device=dev, generator=gen).to(dtype)
    x, before = wide[:, 1:f + 1], wide.clone()
    w, b = torch.randn(nw, device=dev, generator=gen), torch.randn(nb, device=dev, generator=gen)
    y, st = _call(spec, x, w, b)
    got, st2 = _call(spec, x, w, b, out=x)
    assert got.data_ptr() == x.data_ptr() and torch.equal(x, y) and torch.equal(st, st2)
    assert torch.equal(wide[:, 0], before[:, 0]) and torch.equal(wide[:, f + 1:], before[:, f + 1:])


def test_norm_optional_arguments(dev):
    for spec in (65, "5x0e+3x1o"):
        rng = np.random.default_rng(1)
        terms, f, nw, nb = _shape(spec)
        x, xr = _rows(rng, 12, f, torch.float32, dev)
        g, gr = _rows(rng, 12, f, torch.float32, dev)
        y, st = _call(spec, x, None, None)
        _near(y, T.norm_forward(xr, terms)[0], 5e-5, "y")
        rx, rw, rb = T.norm_backward(gr, xr, terms)
        full = _grads(spec, g, x, st, None)
        for got, ref in zip(full, (rx, rw, rb)):
            _near(got, ref, 5e-4, "gradient")
        for need in ((), ("x",), ("weight",), ("bias",), ("x", "bias"), ("weight", "bias")):
            some = _grads(spec, g, x, st, None, need=need)
            for name, a, c in zip(("x", "weight", "bias"), some, full):
                assert (a is None) == (name not in need) and (a is None or torch.equal(a, c))


def test_norm_empty(dev):
    for spec in (8, "5x0e+3x1o"):
        terms, f, nw, nb = _shape(spec)
        x = torch.empty(0, f, device=dev)
        y, st = _call(spec, x, None, None)
        assert y.shape == (0, f) and st.shape == (2, 0, len(terms))
        gx, gw, gb = _grads(spec, x, x, st, None)
        assert gx.shape == (0, f) and (gw == 0).all() and (gb == 0).all() and gw.shape == (nw,) and gb.shape == (nb,)


def test_norm_rows_that_are_constant_or_not_finite(dev):
    # a constant row is its bias; a row that holds NaN or infinity is NaN throughout and no
    # other row changes
    for f in (16, 100, 1312, 5000, 40000):
        rng = np.random.default_rng(2)
        x, _ = _rows(rng, 40, f, torch.float32, dev)
        b = torch.linspace(-1, 1, f, device=dev)
        clean, _ = C.layer_norm_forward(x, None, b)
        x[3], x[4] = 2.5, 0.0
        x[7, f // 2], x[9, 1] = float("nan"), float("inf")
        y, st = C.layer_norm_forward(x, None, b)
        assert torch.equal(y[4], b) and (y[3] - b).abs().max() < 1e-3   # 2.5's mean may miss by some u of 2.5, times 1/sqrt(eps)
        assert y[7].isnan().all() and y[9].isnan().all()
        keep = [r for r in range(40) if r not in (3, 4, 7, 9)]
        assert torch.equal(y[keep], clean[keep])
        g, _ = _rows(rng, 40, f, torch.float32, dev)
        gx, gw, gb = C.layer_norm_backward(g, x, st)
        assert gx[7].isnan().all() and gx[keep].isfinite().all() and gb.isfinite().all()


@pytest.mark.parametrize("spec", [7, 13, 14, 41, 100, 1000, 1025, 1312, 5000, 8193, 16385, 40001, "7x0e+5x1o+13x0e",
                                  "3x1e+20000x0e+41x0e"], ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_norm_constant_rows_are_their_bias(dtype, spec, dev):
    # A row of one value c.  The first mean misses c by at most k u c, k = 70 roundings (chain,
    # tree and quotient); x - mean is exact there, and its own mean, which is added to the
    # first, misses by 2 k u of that, far below half an ulp: the mean is c, and y = bias,
    # exactly.  The variance keeps at most 4 k u (k u c)^2, the difference of two equal terms.
    terms, f, nw, nb = _shape(spec)
    values = [100.0, 1000.0, -60000.0, 0.1, 8192.0, 3.0]
    x = torch.zeros(len(values), f, dtype=dtype, device=dev)
    for off, m, d, _, b0 in terms:
        if b0 is not None:
            x[:, off:off + m] = torch.tensor(values, device=dev)[:, None].to(dtype)
    w, b = torch.linspace(0.5, 1.5, nw, device=dev), torch.linspace(-1, 1, nb, device=dev)
    y, st = _call(spec, x, w, b)
    gen = torch.Generator(device=dev).manual_seed(3)
    g = torch.randint(-4, 5, x.shape, device=dev, generator=gen).to(dtype)
    gx, gw, gb = _grads(spec, g, x, st, w)
    for k, (off, m, d, w0, b0) in enumerate(terms):
        if b0 is None:
            continue
        at = slice(off, off + m)
        assert torch.equal(st[0, :, k], x[:, off].float())
        off_by = 4 * U + 2 * (70 * U) ** 3 * x[:, off].double() ** 2 / 1e-5   # of rstd, relative
        assert ((st[1, :, k].double() * 1e-5 ** 0.5 - 1).abs() <= off_by).all()
        assert torch.equal(y[:, at], b[b0:b0 + m].to(dtype).expand(len(values), m))
        assert (gw[w0:w0 + m] == 0).all() and torch.equal(gb[b0:b0 + m], g[:, at].float().sum(0))   # h = 0; small integers
        a = g[:, at].double() * w[w0:w0 + m].double()
        # rstd (a - mean a), |a| <= 6, mean a by some 100 u
        want = ((a - a.mean(1, keepdim=True)) * 1e-5 ** -0.5).cpu().numpy()
        _near(gx[:, at], want, 6 * 100 * U * 1e-5 ** -0.5 + (off_by[:, None].cpu().numpy() + 4 * U) * np.abs(want), "grad_x")


def test_norm_gradient_by_differences(dev):
    for spec in (48, "16x0e+8x1e+16x1o"):
        rng = np.random.default_rng(3)
        terms, f, nw, nb = _shape(spec)
        x, xr = _rows(rng, 20, f, torch.float32, dev)
        g, gr = _rows(rng, 20, f, torch.float32, dev)
        (w, wr), (b, br) = _weights(rng, nw, torch.float32, dev), _weights(rng, nb, torch.float32, dev)
        _, st = _call(spec, x, w, b)
        gx, gw, gb = (t.double().cpu().numpy() for t in _grads(spec, g, x, st, w))
        loss = lambda x, w, b: (T.norm_forward(x, terms, w, b)[0] * gr).sum()  # noqa: E731
        h = 1e-5
        dx, dw, db = rng.normal(size=xr.shape), rng.normal(size=nw), rng.normal(size=nb)
        for got, lo, hi in (((gx * dx).sum(), (xr - h * dx, wr, br), (xr + h * dx, wr, br)),
                            ((gw * dw).sum(), (xr, wr - h * dw, br), (xr, wr + h * dw, br)),
                            ((gb * db).sum(), (xr, wr, br - h * db), (xr, wr, br + h * db))):
            # the sum of up to 1000 gradients each within 1e-4, and the differences' own error
            assert abs(got - (loss(*hi) - loss(*lo)) / (2 * h)) < 1e-4 * 1000 ** 0.5 + 1e-5 * abs(got)


def test_norm_repeats_bitwise_on_another_stream(dev):
    rng = np.random.default_rng(4)
    x, _ = _rows(rng, 3000, 480, torch.float32, dev)
    g, _ = _rows(rng, 3000, 480, torch.float32, dev)
    y, st = C.layer_norm_forward(x)
    first = (y, *C.layer_norm_backward(g, x, st))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2, st2 = C.layer_norm_forward(x)
        again = (y2, *C.layer_norm_backward(g, x, st2))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, c) for a, c in zip(first, again))


def test_norm_offsets_past_32_bits(dev):
    # rows 2^21 elements apart: the last row's offset is above 2^32 elements
    rows, ld, f = 2100, 1 << 21, 100
    rng = np.random.default_rng(5)
    buf = torch.empty(rows * ld, dtype=torch.bfloat16, device=dev)
    x = buf.view(rows, ld)[:, :f]
    v = torch.from_numpy(rng.normal(size=(rows, f))).to(torch.bfloat16).to(dev)
    x.copy_(v)
    y, st = C.layer_norm_forward(x)
    dense, st2 = C.layer_norm_forward(v)
    assert torch.equal(y, dense) and torch.equal(st, st2)
    got, ref = C.layer_norm_backward(x, x, st), C.layer_norm_backward(v, v, st)
    assert all(torch.equal(a, c) for a, c in zip(got, ref))


def test_norm_in_a_graph(dev):
    rng = np.random.default_rng(6)
    x, _ = _rows(rng, 100, 96, torch.float32, dev)
    g, _ = _rows(rng, 100, 96, torch.float32, dev)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=dev)
    C.layer_norm_backward(g, x, C.layer_norm_forward(x)[1], workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, st = C.layer_norm_forward(x)
        grads = C.layer_norm_backward(g, x, st, workspace=ws)
    for _ in range(4):
        x.copy_(_rows(rng, 100, 96, torch.float32, dev)[0])
        graph.replay()
        torch.cuda.synchronize()
        want, st2 = C.layer_norm_forward(x)
        assert torch.equal(y, want)
        assert all(torch.equal(a, c) for a, c in zip(grads, C.layer_norm_backward(g, x, st2)))


def test_norm_argument_checks(dev):
    x = torch.zeros(4, 8, device=dev)
    st = torch.zeros(2, 4, device=dev)
    bad = [lambda: C.layer_norm_forward(x.double()), lambda: C.layer_norm_forward(x, torch.zeros(8, device=dev).half()),
           lambda: C.layer_norm_forward(x, torch.zeros(8)), lambda: C.layer_norm_forward(x, out=x.bfloat16()),
           lambda: C.layer_norm_backward(x.bfloat16(), x, st), lambda: C.layer_norm_backward(x, x, st.double())]
    for f in bad:
        with pytest.raises(TypeError):
            f()
    bad = [lambda: C.layer_norm_forward(x, torch.zeros(7, device=dev)), lambda: C.layer_norm_forward(x.view(2, 2, 8)),
           lambda: C.layer_norm_forward(x.t()), lambda: C.layer_norm_forward(x[:1].expand(4, 8)),
           lambda: C.layer_norm_forward(x, out=x[:2]), lambda: C.layer_norm_backward(x[:2], x, st),
           lambda: C.layer_norm_backward(x, x, st.t()), lambda: C.irreps_norm_forward(C.NormPlan("9x0e"), x)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(C.CgtpError) as e:
        C.layer_norm_forward(x, eps=-1.0)
    assert e.value.code == -1
    with pytest.raises(C.CgtpError) as e:
        many, st = torch.zeros(1000, 8, device=dev), torch.zeros(2, 1000, device=dev)
        C.layer_norm_backward(many, many, st, workspace=torch.empty(0, dtype=torch.uint8, device=dev))
    assert e.value.code == -5


# ---- AdamW ---------------------------------------------------------------------------

SIZES = [[1], [63, 64, 65], [0, 5, 0, 128, 0], [4095, 4096, 4097, 3], [100000, 1, 17, 8191],
         [(37 * k) % 90 for k in range(500)]]
HYPER = dict(lr=0.02, betas=(0.9, 0.99), eps=1e-6)


def _tensors(rng, sizes, dtype, dev, scale=1.0, skip=0):
    """Tensors that start `skip` elements into their storage."""
    out = []
    for n in sizes:
        t = torch.empty(n + skip, dtype=dtype, device=dev)[skip:]
        out.append(t.copy_(torch.from_numpy(scale * rng.normal(size=n))))
    return out


def _flat(s, tensors):
    """The tensors' values at their places among the states (0 between them), fp32."""
    v = np.zeros(s.state_elems, dtype=np.float32)
    for t, o in zip(tensors, s.offsets):
        v[o:o + t.numel()] = t.float().cpu().numpy()
    return v


def _split(s, v):
    return [v[o:o + n] for n, o in zip(s.sizes, s.offsets)]


def _bits(t):
    return np.ascontiguousarray(t.detach().cpu().numpy()).view(np.uint8)


@pytest.mark.parametrize("pt,gt,skip", [(torch.float32, torch.float32, 0), (torch.float32, torch.bfloat16, 1),
                                        (torch.bfloat16, torch.bfloat16, 0), (torch.float16, torch.float16, 3),
                                        (torch.bfloat16, torch.float32, 1)])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: str(len(s)))
def test_adamw_steps_bitwise(sizes, bits, pt, gt, skip, dev):
    """Three steps from zero states equal the documented fp32 operations bit for bit: params,
    moments, codes and exponents."""
    rng = np.random.default_rng(sum(sizes))
    decay = [0.0 if k % 2 else 0.03 for k in range(len(sizes))]
    s = C.ParamSet(sizes, decay)
    p = _tensors(rng, sizes, pt, dev, skip=skip)
    state = C.adamw_state(s, bits)
    n = s.state_elems
    pr, dr = _flat(s, p), np.repeat(0.0, n)
    for o, c, d in zip(s.offsets, sizes, decay):
        dr[o:o + c] = d
    m, v = np.zeros(n, np.float32), np.zeros(n, np.float32)
    codes = [np.zeros(k, np.uint8) for k in (n, n, n // 64, n // 64)]
    kept = {d: np.float32(1 - HYPER["lr"] * d) for d in (0.0, 0.03)}
    scale = torch.tensor([0.25], device=dev)
    inside = np.zeros(n, bool)
    for o, c in zip(s.offsets, sizes):
        inside[o:o + c] = True
    for t in (1, 2, 3):
        g = _tensors(rng, sizes, gt, dev, scale=10.0 ** rng.uniform(-4, 1), skip=skip)
        C.adamw_step(s, p, g, state, step=t, grad_scale=scale, seed=77 * t, **HYPER)
        if bits == 8:
            m, v = T.decode(codes[0], codes[2], True).astype(np.float32), T.decode(codes[1], codes[3], False).astype(np.float32)
            v = v * v
        base = pr * np.where(dr > 0, kept[0.03], kept[0.0]).astype(np.float32)
        q, m, v, root = T.adamw_f32(base, _flat(s, g), m, v, HYPER["lr"], *HYPER["betas"], HYPER["eps"], t, 0.0, 0.25)
        q = np.where(inside, q, 0).astype(np.float32)
        if bits == 8:
            h = T.random_bits(np.arange(n), 77 * t)
            (codes[0], codes[2]), (codes[1], codes[3]) = T.encode(m, h & 0xffff, True), T.encode(root, h >> 16, False)
        pr = torch.from_numpy(q).to(pt).float().numpy()
        for a, b in zip(p, _split(s, pr)):
            assert np.array_equal(a.float().cpu().numpy(), b), (t, np.abs(a.float().cpu().numpy() - b).max())
        if bits == 32:
            assert np.array_equal(state[0].cpu().numpy(), m) and np.array_equal(state[1].cpu().numpy(), v)
        else:
            for name, a, b in zip(("m", "r", "m exponents", "r exponents"), state, codes):
                assert np.array_equal(a.cpu().numpy(), b), (t, name, (a.cpu().numpy() != b).sum())
            vm, vr = C.adamw_moments(s, state)
            assert np.array_equal(vm.double().cpu().numpy(), T.decode(codes[0], codes[2], True))
            assert np.array_equal(vr.double().cpu().numpy(), T.decode(codes[1], codes[3], False))


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-20, 1e10, 1e17])
def test_adamw8_codes_of_extreme_moments(size, dev):
    # the block exponent spans fp32's range, subnormal moments and vanishing squares included
    rng = np.random.default_rng(13)
    s = C.ParamSet([1000])
    p, state = _tensors(rng, [1000], torch.float32, dev), C.adamw_state(s, 8)
    n = s.state_elems
    codes = [np.zeros(k, np.uint8) for k in (n, n, n // 64, n // 64)]
    pr = _flat(s, p)
    for t in (1, 2, 3):
        g = _tensors(rng, [1000], torch.float32, dev, scale=size)
        C.adamw_step(s, p, g, state, lr=1e-2, step=t, seed=t)
        m, v = T.decode(codes[0], codes[2], True).astype(np.float32), T.decode(codes[1], codes[3], False).astype(np.float32)
        pr, m, _, root = T.adamw_f32(pr, _flat(s, g), m, v * v, 1e-2, 0.9, 0.999, 1e-8, t)
        h = T.random_bits(np.arange(n), t)
        (codes[0], codes[2]), (codes[1], codes[3]) = T.encode(m, h & 0xffff, True), T.encode(root, h >> 16, False)
        for name, a, b in zip(("m", "r", "m exponents", "r exponents"), state, codes):
            assert np.array_equal(a.cpu().numpy(), b), (t, name, (a.cpu().numpy() != b).sum())
        assert np.array_equal(_flat(s, p)[:1000], pr[:1000])


def test_adamw8_rounds_by_the_seed(dev):
    g = [torch.randn(6400, device=dev, generator=torch.Generator(device=dev).manual_seed(0))]
    s = C.ParamSet([6400])
    got = []
    for seed in (1, 1, 2, -3, (1 << 32) + 1):
        state = C.adamw_state(s, 8)
        C.adamw_step(s, [torch.zeros(6400, device=dev)], g, state, lr=1e-2, step=1, seed=seed)
        got.append(state)
    same = [[torch.equal(a, b) for a, b in zip(got[0], q)] for q in got]
    assert all(same[1]) and all(same[4])               # the seed's low 32 bits
    for q in (same[2], same[3]):
        assert q == [False, False, True, True]         # exponents do not hang on it
    # between two seeds' codes lies at most one step
    d = (got[0][1].int() - got[2][1].int()).abs()
    assert d.max() == 1 and 0.2 < (d > 0).float().mean() < 0.5   # two draws differ with probability 2 f (1 - f), a third on average


def test_adamw_against_64_bits(dev):
    rng = np.random.default_rng(8)
    sizes = [5000, 77]
    s = C.ParamSet(sizes, 0.1)
    p, state = _tensors(rng, sizes, torch.float32, dev), C.adamw_state(s)
    pr, m, v = _flat(s, p).astype(np.float64), 0.0, 0.0
    for t in range(1, 21):
        g = _tensors(rng, sizes, torch.float32, dev, scale=1e-3)
        C.adamw_step(s, p, g, state, lr=1e-2, step=t)
        pr, m, v = T.adamw(pr, _flat(s, g), m, v, 1e-2, 0.9, 0.999, 1e-8, t, 0.1)
    # 20 steps, each a rounding of p (|p| < 5) and of an update of at most 0.1 by some 10 u
    assert np.abs(_flat(s, p) - pr).max() < 20 * (5 * U * 2 + 0.1 * 20 * U)


def test_adamw8_follows_adamw32(dev):
    # the same gradients with both states: the 8-bit run's path stays near the 32-bit one's, in
    # both directions of the second moment (the gradients shrink a hundredfold half-way)
    rng = np.random.default_rng(9)
    s = C.ParamSet([20000])
    p32, p8 = [torch.zeros(20000, device=dev)], [torch.zeros(20000, device=dev)]
    st32, st8 = C.adamw_state(s), C.adamw_state(s, 8)
    sign = torch.from_numpy(np.where(rng.random(20000) < 0.5, -1.0, 1.0)).float().to(dev)
    size = torch.from_numpy(10.0 ** rng.uniform(-2, 0, 20000)).float().to(dev)
    for t in range(1, 601):
        g = [(sign + torch.from_numpy(rng.normal(size=20000)).float().to(dev)) * size * (1.0 if t <= 300 else 0.01)]
        C.adamw_step(s, p32, g, st32, lr=1e-3, betas=(0.9, 0.99), step=t)
        C.adamw_step(s, p8, g, st8, lr=1e-3, betas=(0.9, 0.99), step=t, seed=t)
    # a code's distance is 2^-3 of m and 2^-4 of r; held over 1/(1 - b) steps the roundings'
    # deviations stay below one distance, so single updates differ by a quarter and, being
    # unbiased, their sum over hundreds of steps by far less
    rel = (p8[0] - p32[0]).norm() / p32[0].norm()
    assert rel < 0.1, rel
    _, r = C.adamw_moments(s, st8)
    r32 = st32[1].sqrt()
    assert abs((r.float()[:20000] / r32[:20000]).mean() - 1) < 0.05


@pytest.mark.parametrize("place", range(4))
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 1e30])
def test_adamw8_moments_that_are_not_finite_leave_their_block_alone(bad, place, dev):
    # one such gradient at each place of a lane's four, beside zeros, small values and the
    # block's largest (1e30: the square overflows, the first moment does not): codes and
    # exponents of the whole block equal the reference's, then and in the step after
    rng = np.random.default_rng(15)
    n = 64 * 48
    s = C.ParamSet([n])
    p, state = _tensors(rng, [n], torch.float32, dev), C.adamw_state(s, 8)
    codes = [np.zeros(k, np.uint8) for k in (n, n, n // 64, n // 64)]
    pr = _flat(s, p)
    for t in (1, 2, 3):
        v = rng.normal(size=n) * np.where(rng.random(n) < 0.3, 1e-3, 1.0) * (rng.random(n) < 0.7)
        if t > 1:
            for k in range(48):   # every block: beside a zero, a small value, the largest
                at = 64 * k + 4 * (k % 16) + place
                near = 64 * k + (at + 1 if k % 2 else at - 1) % 64
                v[near] = (0.0, 1e-3, 4.0)[k % 3]
                if t == 2:
                    v[at] = bad
        g = [torch.from_numpy(v).float().to(dev)]
        C.adamw_step(s, p, g, state, lr=1e-2, step=t, seed=t)
        m, v = T.decode(codes[0], codes[2], True).astype(np.float32), T.decode(codes[1], codes[3], False).astype(np.float32)
        pr, m, _, root = T.adamw_f32(pr, _flat(s, g), m, v * v, 1e-2, 0.9, 0.999, 1e-8, t)
        assert t == 1 or (~np.isfinite(root)).sum() == 48
        h = T.random_bits(np.arange(n), t)
        (codes[0], codes[2]), (codes[1], codes[3]) = T.encode(m, h & 0xffff, True), T.encode(root, h >> 16, False)
        got = [a.cpu().numpy() for a in state]
        codes[0][codes[0] == 128] = got[0][got[0] == 128] = 0   # a zero's sign is free
        for name, a, b in zip(("m", "r", "m exponents", "r exponents"), got, codes):
            assert np.array_equal(a, b), (t, name, (a != b).sum())
        assert np.array_equal(_flat(s, p), pr, equal_nan=True)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_skips_on_nan_scale_and_contains_bad_gradients(bits, dev):
    rng = np.random.default_rng(10)
    sizes = [300, 70]
    s = C.ParamSet(sizes, 0.1)
    p, g, state = _tensors(rng, sizes, torch.float32, dev), _tensors(rng, sizes, torch.float32, dev), C.adamw_state(s, bits)
    C.adamw_step(s, p, g, state, lr=1e-2, step=1)
    before = [t.clone() for t in (*p, *state)]
    C.adamw_step(s, p, g, state, lr=1e-2, step=2, grad_scale=torch.tensor([float("nan")], device=dev))
    assert all(torch.equal(a, b) for a, b in zip(before, (*p, *state)))
    g[0][10], g[0][100], g[1][69] = float("nan"), float("inf"), -float("inf")
    clean = [t.clone() for t in (*p, *state)]
    g2 = [torch.nan_to_num(t, 0.0, 0.0, 0.0) for t in g]
    C.adamw_step(s, clean[:2], g2, tuple(clean[2:]), lr=1e-2, step=2)
    C.adamw_step(s, p, g, state, lr=1e-2, step=2)
    hit = torch.zeros(300, dtype=torch.bool, device=dev)
    hit[[10, 100]] = True
    assert p[0][hit].isnan().all() and torch.equal(p[0][~hit], clean[0][~hit])
    assert p[1][69].isnan() and torch.equal(p[1][:69], clean[1][:69])
    if bits == 8:
        m, r = C.adamw_moments(s, state)
        assert m[10].isnan() and r[10].isnan() and m[100].isnan() and r[100].isnan()
        assert m.isnan().sum() == 3 and r.isnan().sum() == 3


def test_adamw_repeats_bitwise_and_in_a_graph(dev):
    rng = np.random.default_rng(11)
    sizes = [5000, 33, 700]
    s = C.ParamSet(sizes)
    g = s.pointers(_tensors(rng, sizes, torch.float32, dev))
    start = _tensors(rng, sizes, torch.float32, dev)

    def fresh():
        return [t.clone() for t in start], C.adamw_state(s, 8)

    def step(p, st):
        f = C.grad_norm(s, g, 1.0)
        C.adamw_step(s, p, g, st, lr=1e-2, step=3, grad_scale=f[1:], seed=5)
        return f

    p, st = fresh()
    for _ in range(3):
        norm = step(p, st)
    q, su = fresh()
    step(*fresh())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm2 = step(q, su)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*p, *st, norm), (*q, *su, norm2)))


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_set_that_outgrows_the_cache(bits, dev):
    # more than 256 MB: each tensor is what it is in a set of its own, bit for bit (8-bit states
    # round by their place in the set: the last tensor's are checked against the reference)
    sizes = [9000001, 5, 8000000]
    gen = torch.Generator(device=dev).manual_seed(0)
    p, g = ([torch.randn(n, device=dev, generator=gen) for n in sizes] for _ in range(2))
    start, s = [t.clone() for t in p], C.ParamSet(sizes, 0.1)
    state = C.adamw_state(s, bits)
    C.adamw_step(s, p, g, state, lr=1e-2, step=1, seed=9)
    for k, n in enumerate(sizes):
        one, alone = C.ParamSet([n], 0.1), [start[k]]
        st = C.adamw_state(one, bits)
        C.adamw_step(one, alone, [g[k]], st, lr=1e-2, step=1, seed=9)
        assert torch.equal(alone[0], p[k])
        if bits == 32:
            at = slice(s.offsets[k], s.offsets[k] + n)
            assert all(torch.equal(a[at], b[:n]) for a, b in zip(state, st))
    if bits == 8:
        n = 64 * 1000
        at = s.offsets[2] + sizes[2] - n
        zero = np.zeros(n, np.float32)
        _, m, _, root = T.adamw_f32(zero, g[2][-n:].cpu().numpy(), zero, zero, 1e-2, 0.9, 0.999, 1e-8, 1)
        h = T.random_bits(np.arange(at, at + n), 9)
        for values, u, signed, c, e in ((m, h & 0xffff, True, state[0], state[2]), (root, h >> 16, False, state[1], state[3])):
            code, exp = T.encode(values, u, signed)
            assert np.array_equal(c[at:at + n].cpu().numpy(), code)
            assert np.array_equal(e[at // 64:(at + n) // 64].cpu().numpy(), exp)


@pytest.mark.parametrize("pt,gt", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32), (torch.float32, torch.float16)])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_past_the_cache_in_16_bits(bits, pt, gt, dev):
    # as above, 16-bit parameters and gradients: parameters as in sets of their own, and the states
    # of the first tensor, whose places are the same there
    sizes = [30000001, 7, 9000000] if bits == 8 else [12000001, 7, 4000000]
    gen = torch.Generator(device=dev).manual_seed(0)
    p = [torch.randn(n, device=dev, generator=gen).to(pt) for n in sizes]
    g = [torch.randn(n, device=dev, generator=gen).to(gt) for n in sizes]
    start, s = [t.clone() for t in p], C.ParamSet(sizes, 0.1)
    state = C.adamw_state(s, bits)
    C.adamw_step(s, p, g, state, lr=1e-2, step=1, seed=9)
    for k, n in enumerate(sizes):
        for from_, to in ((0, n // 3), (n // 3, n)):   # in pieces that stay in the cache
            one, alone = C.ParamSet([to - from_], 0.1), [start[k][from_:to].clone()]
            st = C.adamw_state(one, bits)
            C.adamw_step(one, alone, [g[k][from_:to].clone()], st, lr=1e-2, step=1, seed=9)
            assert torch.equal(alone[0], p[k][from_:to])
            if k == 0 and from_ == 0:
                m = (to - from_) // 64 * 64
                assert all(torch.equal(a[:m], c[:m]) for a, c in zip(state[:2], st[:2]))
                assert all(torch.equal(a[:m // 64], c[:m // 64]) for a, c in zip(state[2:], st[2:]))


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_counts_on_the_device(bits, dev):
    # steps counted on the device equal the host's bit for bit, eager and replayed in a graph; a
    # skipped step does not count; the rate may change between replays
    rng = np.random.default_rng(14)
    sizes = [3000, 70]
    s = C.ParamSet(sizes, 0.1)
    start = _tensors(rng, sizes, torch.float32, dev)
    p, q = [t.clone() for t in start], [t.clone() for t in start]
    g = s.pointers([torch.empty(n, device=dev) for n in sizes])
    st, su = C.adamw_state(s, bits), C.adamw_state(s, bits)
    count = torch.zeros(1, dtype=torch.int64, device=dev)
    lr, scale = torch.empty(1, device=dev), torch.ones(1, device=dev)

    def step():
        C.adamw_step(s, q, g, su, lr=lr, betas=(0.9, 0.99), step=count, grad_scale=scale, seed=5)

    def same():
        assert all(torch.equal(a, b) for a, b in zip((*p, *st), (*q, *su)))

    def draw():
        for t in g.tensors:
            t.copy_(torch.from_numpy(rng.normal(size=t.numel())))

    graph = None
    for t in range(1, 8):
        draw()
        rate = 1e-2 / t
        lr.fill_(rate)
        C.adamw_step(s, p, g, st, lr=float(np.float32(rate)), betas=(0.9, 0.99), step=t, grad_scale=scale, seed=5 + t)
        if t == 4:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        if graph is None:
            step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        same()
        assert int(count) == t
        if t == 5:
            scale.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            same()
            assert int(count) == t
            scale.fill_(1.0)
    for bad in (dict(lr=1.0, step=count.int()), dict(lr=lr.double(), step=count), dict(lr=1.0, step=count.cpu())):
        with pytest.raises(TypeError):
            C.adamw_step(s, q, g, su, **bad)


def test_adamw_tensor_past_32_bits(dev):
    # one tensor of 2^32 + 1000 elements in bf16 with 8-bit states: its last elements move as
    # those of a small one at the same places, and the first ones too
    n = (1 << 32) + 1000
    s = C.ParamSet([n])
    p, g = [torch.ones(n, dtype=torch.bfloat16, device=dev)], [torch.zeros(n, dtype=torch.bfloat16, device=dev)]
    g[0][-500:], g[0][:500] = 1.0, -1.0
    state = C.adamw_state(s, 8)
    C.adamw_step(s, p, g, state, lr=0.25, step=1)
    assert (p[0][-500:] == 0.75).all() and (p[0][:500] == 1.25).all() and (p[0][500:-500] == 1).all()
    f = C.grad_norm(s, g)
    assert abs(float(f[0]) - 1000 ** 0.5) < 1e-4 and float(f[1]) == 1.0


@pytest.mark.parametrize("gt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: str(len(s)))
def test_grad_norm(sizes, gt, dev):
    rng = np.random.default_rng(12)
    s = C.ParamSet(sizes)
    g = _tensors(rng, sizes, gt, dev, skip=1)
    scale = torch.tensor([0.5], device=dev)
    for most in (float("inf"), 1e-2, 1e9):
        norm, factor = T.grad_norm([t.double().cpu().numpy() for t in g], 0.5, most)
        got = C.grad_norm(s, g, most, grad_scale=scale).double().cpu().numpy()
        assert abs(got[0] - norm) <= 2 * U * norm and abs(got[1] - factor) <= 4 * U * factor


def test_grad_norm_extremes(dev):
    s = C.ParamSet([100, 50])
    zero = [torch.zeros(100, device=dev), torch.zeros(50, device=dev)]
    assert C.grad_norm(s, zero, 1.0).tolist() == [0.0, 1.0]
    huge = [torch.full((100,), 1e30, device=dev), zero[1]]
    got = C.grad_norm(s, huge, 1.0).tolist()
    assert abs(got[0] / 1e31 - 1) < 1e-6 and abs(got[1] / 1e-31 - 1) < 1e-6
    tiny = [torch.full((100,), 1e-30, device=dev), zero[1]]
    assert abs(C.grad_norm(s, tiny).tolist()[0] / 1e-29 - 1) < 1e-6
    for bad in (float("nan"), float("inf")):
        zero[1][49] = bad
        assert np.isnan(C.grad_norm(s, zero, 1.0).tolist()[1])
    assert C.grad_norm(C.ParamSet([]), [], 1.0).tolist() == [0.0, 1.0]


def test_optimiser_argument_checks(dev):
    s = C.ParamSet([4, 6])
    p, g, st = [torch.zeros(4, device=dev), torch.zeros(6, device=dev)], [torch.zeros(4, device=dev), torch.zeros(6, device=dev)], C.adamw_state(s)
    for kw in (dict(lr=-1.0), dict(lr=float("nan")), dict(lr=1.0, betas=(1.0, 0.9)), dict(lr=1.0, betas=(0.9, -0.1)),
               dict(lr=1.0, eps=-1.0), dict(lr=1.0, step=0)):
        with pytest.raises(C.CgtpError) as e:
            C.adamw_step(s, p, g, st, **kw)
        assert e.value.code == -1
    with pytest.raises(C.CgtpError):
        C.grad_norm(s, g, max_norm=0.0)
    with pytest.raises(C.CgtpError) as e:
        C.grad_norm(C.ParamSet([100000]), [torch.zeros(100000, device=dev)],
                    workspace=torch.empty(0, dtype=torch.uint8, device=dev))
    assert e.value.code == -5
    for f in (lambda: s.pointers(p[:1]), lambda: s.pointers([p[1], p[0]]), lambda: s.pointers([p[0], torch.zeros(6, 2, device=dev)[:, 0]]),
              lambda: C.adamw_step(s, p, g, st[:1], lr=1.0), lambda: C.adamw_step(s, p, g, (st[0], st[1][:-1]), lr=1.0)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: s.pointers([p[0], p[1].half()]), lambda: s.pointers([p[0], p[1].cpu()]),
              lambda: C.adamw_step(s, p, g, (st[0], st[1].double()), lr=1.0),
              lambda: C.adamw_step(s, p, g, st, lr=1.0, grad_scale=torch.zeros(1))):
        with pytest.raises(TypeError):
            f()
    assert all((t == 0).all() for t in (*p, *st))


def test_workspaces_are_contiguous(dev):
    # an expanded or strided tensor has more elements than the memory that follows its address
    x = torch.zeros(1000, 8, device=dev)
    _, st = C.layer_norm_forward(x)
    p, s = C.NormPlan("8x0e"), C.ParamSet([100000])
    _, sti = C.irreps_norm_forward(p, x)
    one = torch.empty(1, dtype=torch.uint8, device=dev)
    for ws in (one.expand(1 << 20), torch.empty(1 << 20, 2, dtype=torch.uint8, device=dev)[:, 0]):
        for f in (lambda: C.layer_norm_backward(x, x, st, workspace=ws),
                  lambda: C.irreps_norm_backward(p, x, x, sti, workspace=ws),
                  lambda: C.grad_norm(s, [torch.zeros(100000, device=dev)], workspace=ws)):
            with pytest.raises(ValueError):
                f()
    for f in (lambda: C.layer_norm_backward(x, x, st, workspace=one.cpu()), lambda: C.layer_norm_backward(x, x, st, workspace=7)):
        with pytest.raises(TypeError):
            f()


def test_layouts_keep_their_memory_and_notice_other_tensors_memory(dev):
    # laid out once, then tensors are given other memory: a call neither reads nor writes memory
    # that was freed, and where all have moved it is refused
    s = C.ParamSet([300, 70, 1])

    def fresh():
        p, g = ([torch.ones(n, device=dev) for n in s.sizes] for _ in range(2))
        return p, g, C.adamw_state(s), s.pointers(p), s.pointers(g)

    changes = (lambda t: setattr(t, "data", torch.ones(t.shape, device=dev)), lambda t: t.set_(torch.ones(t.shape, device=dev)))
    for change in changes:
        for which in ((0,), (2,), (0, 1, 2)):
            p, g, state, laid, grads = fresh()
            for k in which:
                change(p[k])
                change(g[k])
            for f in (lambda: C.adamw_step(s, laid, g, state, lr=1e-2, step=1), lambda: C.grad_norm(s, grads),
                      lambda: C.adamw_step(s, p, grads, state, lr=1e-2, step=1)):
                with pytest.raises(ValueError, match="other memory"):
                    f()
            assert all((t == 1).all() for t in p) and all((t == 0).all() for t in state)
            C.adamw_step(s, s.pointers(p), s.pointers(g), state, lr=1e-2, step=1)
            assert all((t < 1).all() for t in p)
        # one between them: the layout goes on with the memory that it keeps
        p, g, state, laid, grads = fresh()
        at = p[1].data_ptr()
        change(p[1])
        others = [torch.full((70,), 5.0, device=dev) for _ in range(50)]   # would reuse freed memory
        assert at not in [t.data_ptr() for t in others]
        C.adamw_step(s, laid, grads, state, lr=1e-2, step=1)
        assert (p[1] == 1).all() and all((t == 5).all() for t in others) and (p[0] < 1).all()
