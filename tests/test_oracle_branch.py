"""Pins of the fp64 references of the operators for branching networks: each against
something other than itself."""
import numpy as np
import pytest

import oracle as O
import workloads as WL
from oracle import branch_oracle as B


@pytest.mark.parametrize("act", [None, "silu", "gelu"])
def test_activation_slopes(act):
    z = np.linspace(-6, 6, 101)
    h = 1e-6
    diff = (B.activation(z + h, act)[0] - B.activation(z - h, act)[0]) / (2 * h)
    assert np.abs(diff - B.activation(z, act)[1]).max() < 1e-8


def test_group_norm_standardises():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(40, 12)) * 3 + 5
    off = [0, 7, 7, 30, 36]
    y, mean, rstd = B.group_norm_forward(x, 3, off, eps=0.0)
    for lo, hi in ((0, 7), (7, 30), (30, 36)):
        for g in range(3):
            q = y[lo:hi, 4 * g:4 * g + 4]
            assert abs(q.mean()) < 1e-12 and abs((q ** 2).mean() - 1) < 1e-12
    assert (y[36:] == 0).all() and mean[1].tolist() == [0, 0, 0] and np.isinf(rstd[1]).all()
    # one group of a one-row sample is a layer norm
    y, _, _ = B.group_norm_forward(x, 1, list(range(41)))
    assert np.allclose(y, (x - x.mean(1, keepdims=True)) / np.sqrt(x.var(axis=1, keepdims=True) + 1e-5))


@pytest.mark.parametrize("act", [None, "silu", "gelu"])
def test_group_norm_gradients(act):
    rng = np.random.default_rng(1)
    x, g = rng.normal(size=(20, 6)), rng.normal(size=(20, 6))
    w, b = rng.normal(size=6), rng.normal(size=6)
    off = [2, 5, 18]
    gx, gw, gb = B.group_norm_backward(g, x, 2, off, w, b, act)
    loss = lambda x, w, b: (B.group_norm_forward(x, 2, off, w, b, act)[0] * g).sum()  # noqa: E731
    h = 1e-6
    for got, k in ((gx, 0), (gw, 1), (gb, 2)):
        args = [x, w, b]
        for at in np.ndindex(got.shape):
            d = np.zeros_like(args[k])
            d[at] = h
            up, down = list(args), list(args)
            up[k], down[k] = args[k] + d, args[k] - d
            assert abs((loss(*up) - loss(*down)) / (2 * h) - got[at]) < 1e-7
    assert (gx[:2] == 0).all() and (gx[18:] == 0).all()


def test_route_by_a_loop():
    rng = np.random.default_rng(2)
    z = np.round(rng.normal(size=(60, 7)) * 2) / 2   # ties
    z[3], z[5, :5], z[9, 2] = -np.inf, -np.inf, -np.inf
    mask = rng.random(60) < 0.7
    ids, gates, counts, balance, slope = B.route_forward(z, 3, mask, renormalise=True)
    want, total, prob, part = np.zeros(7, int), 0.0, np.zeros(7), 0
    for r in range(60):
        left = [e for e in range(7) if z[r, e] > -np.inf] if mask[r] else []
        picks = []
        for _ in range(3):
            if left:
                best = max(left, key=lambda e: (z[r, e], -e))
                left.remove(best)
                picks.append(best)
        assert ids[r].tolist() == picks + [-1] * (3 - len(picks))
        if picks:
            part += 1
            e = np.exp(z[r] - z[r].max())
            prob += e / e.sum()
            q = np.exp(z[r, picks] - z[r].max())
            assert np.allclose(gates[r, :len(picks)], q / q.sum())
        assert (gates[r, len(picks):] == 0).all()
        for e in picks:
            want[e] += 1
    assert counts.tolist() == want.tolist()
    assert np.isclose(balance, 7 * (want / want.sum() * prob / part).sum())


def test_balance_closed_forms():
    n = 5
    even = 30.0 * np.eye(n)[np.arange(100) % n]
    assert np.isclose(B.route_forward(even, 1)[3], 1.0)
    one = np.zeros((100, n))
    one[:, 2] = 60.0
    assert np.isclose(B.route_forward(one, 1)[3], n)
    assert B.route_forward(np.zeros((4, n)), 1, np.zeros(4))[3] == 0.0


@pytest.mark.parametrize("renormalise", [False, True])
def test_route_gradient(renormalise):
    rng = np.random.default_rng(3)
    z, up = rng.normal(size=(8, 6)), rng.normal(size=(8, 3))
    mask = np.arange(8) != 4
    ids, _, _, _, slope = B.route_forward(z, 3, mask, renormalise)
    got = B.route_backward(z, ids, slope, up, 1.7, renormalise)

    def loss(z):
        p = B.softmax(z) * mask[:, None]
        q = np.take_along_axis(p, np.maximum(ids, 0), 1) * (ids >= 0)
        if renormalise:
            q = q / np.maximum(q.sum(1, keepdims=True), 1e-300)
        return (q * up).sum() + 1.7 * (p * slope).sum()

    h = 1e-6
    for at in np.ndindex(z.shape):
        d = np.zeros_like(z)
        d[at] = h
        assert abs((loss(z + d) - loss(z - d)) / (2 * h) - got[at]) < 1e-7


def test_gate_gradient_is_the_convolutions():
    wl = WL.WORKLOADS["tiny"]
    pos, box, cell, rng = WL.positions(wl)
    rp, col, sh = O.neighbors(pos, box, wl.cutoff)
    plan = O.build_plan(wl.irreps_in, wl.irreps_sh, wl.l_out_max, wl.rule)
    x, w, _ = WL.draw_payload(wl, rng, wl.n_atoms, plan.f_in, len(col), plan.w_per_edge)
    w = w.astype(np.float64)
    gate = np.where(rng.random(len(col)) < 0.3, 0.0, 1 - rng.random(len(col)))
    up = rng.normal(size=(wl.n_atoms, plan.f_out))
    mask = (np.arange(len(col)) % 5 != 0).astype(np.uint8)
    # the message is linear in gate w: dL/dw of the gated convolution is the gate times the plain one's
    plain = O.conv_backward(plan, pos, cell, rp, col, sh, x, w, up, mask)[1]
    got = B.gate_backward(w, plain * gate[:, None], gate, mask)
    loss = lambda f: (O.conv_forward(plan, pos, cell, rp, col, sh, x, w * f[:, None], mask) * up).sum()  # noqa: E731
    for e in np.nonzero((gate != 0) & (mask != 0))[0][::17]:
        d = np.zeros(len(col))
        d[e] = 1e-3   # linear: any step
        assert abs((loss(gate + d) - loss(gate - d)) / 2e-3 - got[e]) < 1e-8 * max(1.0, abs(got[e]))
    assert (got[gate == 0] == 0).all() and (got[mask == 0] == 0).all()
