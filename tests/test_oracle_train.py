"""CPU pins of the training operators' references (oracle/train_oracle.py)."""
import numpy as np
import pytest

import oracle as O
from oracle import train_oracle as T

IRREPS = "6x0e+4x1o+3x2e+2x0o+1x3o+5x0e"


def _terms(spec):
    return T.row_terms(spec) if isinstance(spec, int) else T.norm_terms(spec)


def _width(terms):
    return sum(m * d for _, m, d, _, _ in terms)


def test_layer_norm_standardises_rows():
    x = np.random.default_rng(0).normal(size=(5, 33)) * 3 + 7
    y, mean, rstd = T.norm_forward(x, T.row_terms(33), eps=0.0)
    np.testing.assert_allclose(y.mean(axis=1), 0, atol=1e-13)
    np.testing.assert_allclose(y.std(axis=1), 1, rtol=1e-13)
    np.testing.assert_allclose(mean[:, 0], x.mean(axis=1), rtol=1e-14)
    np.testing.assert_allclose(rstd[:, 0], 1 / x.std(axis=1), rtol=1e-13)
    one, _, _ = T.norm_forward(x[:, :1], T.row_terms(1), weight=[2.0], bias=[0.5])
    assert np.array_equal(one, np.full((5, 1), 0.5))


@pytest.mark.parametrize("spec", [1, 4, 9, IRREPS])
def test_gradients_by_differences(spec):
    rng = np.random.default_rng(1)
    terms = _terms(spec)
    x, g = rng.normal(size=(4, _width(terms))), rng.normal(size=(4, _width(terms)))
    w, b = rng.normal(size=sum(t[1] for t in terms)), rng.normal(size=sum(t[1] for t in terms if t[4] is not None))
    gx, gw, gb = T.norm_backward(g, x, terms, w)

    def loss(x, w, b):
        return (T.norm_forward(x, terms, w, b)[0] * g).sum()

    h = 1e-5
    for arr, grad, put in ((x, gx, lambda v: (v, w, b)), (w, gw, lambda v: (x, v, b)), (b, gb, lambda v: (x, w, v))):
        for _ in range(6):
            d = rng.normal(size=arr.shape)
            diff = (loss(*put(arr + h * d)) - loss(*put(arr - h * d))) / (2 * h)
            # central differences: h^2 of a third derivative of order rstd^3 ~ 1, and rounding 1e-16/h
            np.testing.assert_allclose((grad * d).sum(), diff, rtol=1e-6, atol=1e-7)


def test_irreps_norm_is_equivariant():
    rng = np.random.default_rng(2)
    terms, ir = T.norm_terms(IRREPS), O.parse_irreps(IRREPS)
    x = rng.normal(size=(3, _width(terms)))
    w, b = rng.normal(size=sum(t[1] for t in terms)), rng.normal(size=11)
    rot = O.random_rotation(rng)

    def act(v, inversion):
        out = v.copy()
        for (off, mul, d, _, _), (_, l, p) in zip(terms, ir):
            q = v[:, off:off + mul * d].reshape(-1, mul, d)
            q = q * p if inversion else q @ O.wigner_d_real(l, rot).T
            out[:, off:off + mul * d] = q.reshape(v.shape[0], -1)
        return out

    for inversion in (False, True):
        np.testing.assert_allclose(T.norm_forward(act(x, inversion), terms, w, b)[0],
                                   act(T.norm_forward(x, terms, w, b)[0], inversion), atol=1e-11)


def test_scalar_irreps_norm_is_the_layer_norm():
    x = np.random.default_rng(3).normal(size=(4, 12))
    a, b = T.norm_forward(x, T.norm_terms("12x0e")), T.norm_forward(x, T.row_terms(12))
    assert all(np.array_equal(u, v) for u, v in zip(a, b))


def test_adamw_closed_form():
    # a constant gradient from zero states: m = (1 - b1^t) g, v = (1 - b2^t) g^2, so that every
    # step moves p by lr g / (|g| + eps) behind its decay
    g, p, m, v = np.array([0.5, -2.0, 1e-3]), np.ones(3), np.zeros(3), np.zeros(3)
    want = p.copy()
    for t in range(1, 6):
        p, m, v = T.adamw(p, g, m, v, 0.1, 0.9, 0.99, 1e-3, t, decay=0.2)
        want = want * (1 - 0.02) - 0.1 * g / (np.abs(g) + 1e-3)
        np.testing.assert_allclose(p, want, rtol=1e-13)
    got = T.adamw_f32(np.ones(3), g, np.zeros(3), np.zeros(3), 0.1, 0.9, 0.99, 1e-3, 1, decay=0.2)
    np.testing.assert_allclose(got[0], T.adamw(np.ones(3), g, np.zeros(3), np.zeros(3), 0.1, 0.9, 0.99, 1e-3, 1, 0.2)[0],
                               rtol=1e-6)


@pytest.mark.parametrize("signed", [True, False])
def test_codes_return_the_grid(signed):
    # every code's own value is stored as that code whatever the random bits (a block whose
    # largest value fills the top octave), and the grid rises
    codes = np.arange(120 if signed else 240, dtype=np.uint8)
    codes = np.concatenate([codes, np.full(-len(codes) % 64, codes[-1])]).reshape(-1, 64)
    codes[:, 0] = codes.max()
    codes = codes.reshape(-1)
    for e in (30, 120, 140):
        v = T.decode(codes, np.full(len(codes) // 64, e, dtype=np.uint8), signed)
        for u in (0, 40000, 65535):
            c, ee = T.encode(v.astype(np.float32), np.full(len(codes), u), signed)
            assert np.array_equal(c, codes) and np.all(ee == e)
    assert np.all(np.diff(T._grid(np.arange(127), 3)) > 0) and np.all(np.diff(T._grid(np.arange(255), 4)) > 0)


@pytest.mark.parametrize("signed", [True, False])
def test_rounding_keeps_the_mean(signed):
    rng = np.random.default_rng(4)
    v = (rng.normal(size=64) * 10.0 ** rng.uniform(-3, 0, size=64)).astype(np.float32)
    v = v if signed else np.abs(v)
    rounds = 4000
    got = np.zeros(64)
    for s in range(rounds):
        h = T.random_bits(np.arange(64), s)
        c, e = T.encode(v, (h & 0xffff) if signed else (h >> 16), signed)
        got += T.decode(c, e, signed)
    # a rounding's deviation is at most half a code's distance (2^-3 or 2^-4 of the value, or of
    # the smallest normal value): five deviations of the mean of 4000
    step = np.maximum(np.abs(v), 2.0 ** np.floor(np.log2(np.abs(v).max())) * 2.0 ** -13) * (2.0 ** -3 if signed else 2.0 ** -4)
    assert np.all(np.abs(got / rounds - v) <= 5 * 0.5 * step / np.sqrt(rounds) + step * 2.0 ** -16)


def test_codes_of_values_that_are_not_finite():
    v = np.ones(64, dtype=np.float32)
    v[3], v[5], v[7] = np.nan, np.inf, 0.0
    for signed, nan in ((True, 127), (False, 255)):
        c, e = T.encode(v, np.zeros(64, dtype=int), signed)
        assert c[3] == nan and c[5] == nan and c[7] == 0 and e[0] == 127
        got = T.decode(c, e, signed)
        assert np.isnan(got[[3, 5]]).all() and np.array_equal(np.delete(got, [3, 5]), np.delete(v, [3, 5]))
    tiny = np.full(64, 1e-9, dtype=np.float32)
    tiny[0] = 1.0
    c, _ = T.encode(tiny, np.zeros(64, dtype=int), False)
    assert np.all(c[1:] == 1)          # a positive root is never stored as 0


def test_random_bits_are_even():
    # 2^20 elements of one step, and 2^16 steps of one element: each 16-bit half in 64 bins,
    # chi-squared with 63 degrees of freedom (mean 63, deviation 11.2) within six deviations;
    # neighbours, halves and successive steps uncorrelated within five deviations
    for h in (T.random_bits(np.arange(1 << 20), 7), np.array([T.random_bits(5, s) for s in range(1 << 16)]),
              T.random_bits(np.arange(1 << 18) + (5 << 32), 123456789)):
        n = h.size
        halves = [(h & np.uint32(0xffff)).astype(float) / 65536, (h >> np.uint32(16)).astype(float) / 65536]
        for u in halves:
            c = np.bincount((u * 64).astype(int), minlength=64)
            assert ((c - n / 64) ** 2 / (n / 64)).sum() < 63 + 6 * 11.3
            for lag in (1, 2, 64):
                assert abs(((u[lag:] - 0.5) * (u[:-lag] - 0.5)).mean() * 12) < 5 / np.sqrt(n - lag)
        assert abs(((halves[0] - 0.5) * (halves[1] - 0.5)).mean() * 12) < 5 / np.sqrt(n)


def test_grad_norm():
    s, f = T.grad_norm([np.array([3.0]), np.array([[4.0]])], scale=2.0, max_norm=5.0)
    assert s == 10 and f == 1.0
    assert T.grad_norm([np.zeros(3)], 0.5, 1.0) == (0.0, 0.5)
    assert np.isnan(T.grad_norm([np.array([np.inf])])[1])
