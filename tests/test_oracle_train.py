"""Pins of the routing and optimizer oracles: closed forms, differences, and the formats."""
import math

import numpy as np
import pytest

from oracle import optim as oo
from oracle import route as orr

GATES = [orr.Gate(12, 3, s, g, tg, gs, r, c)
         for s in ("softmax", "sigmoid") for g, tg, gs in ((1, 1, "max"), (4, 2, "max"), (4, 2, "top2"))
         for r, c in ((True, 2.5), (False, 1.0))]


@pytest.mark.parametrize("gate", GATES, ids=str)
def test_route_gradient_against_differences(gate):
    rng = np.random.default_rng(3)
    x, dw, b = rng.standard_normal((5, 12)), rng.standard_normal((5, 3)), 0.1 * rng.standard_normal(12)
    idx, w, _ = orr.forward(gate, x, b)
    got = orr.backward(gate, x, idx, dw)
    h = 1e-6
    for n in range(5):
        for e in range(12):
            up, down = x[n].copy(), x[n].copy()
            up[e] += h
            down[e] -= h
            of = [int(i) for i in idx[n]]
            d = (dw[n] * (orr.weights_row(gate, up, of) - orr.weights_row(gate, down, of))).sum() / (2 * h)
            # a central difference of a smooth function of size 1: h^2 and 1e-16 / h
            assert abs(d - got[n, e]) <= 1e-8


def test_route_softmax_renormalised_is_softmax_over_the_chosen():
    # the layer's own gate: top-k of the logits, softmax over them
    from oracle import moe_oracle as mo
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 16)).astype(np.float32)
    idx, w, load = orr.forward(orr.Gate(16, 4), x)
    ref_idx, ref_p = mo.topk_gating(x, 4)
    assert np.array_equal(idx, ref_idx) and np.abs(w - ref_p).max() < 1e-14
    assert load.sum() == 160


def test_route_choice_by_hand():
    gate = orr.Gate(8, 2, "sigmoid", 4, 2, "top2", True, 2.5)
    x = np.array([3.0, -9, 1.5, 1.5, 2.9, -9, 0, 0])
    # groups score sigmoid sums .953, 1.635, .948, 1.0: groups 1 and 3 stay although 0 and 2 hold the
    # two largest logits
    assert orr.choose_row(gate, x) == [2, 3]
    # a bias on expert 6 moves it to the front of the choice, and changes no weight
    b = np.zeros(8)
    b[6] = 0.5
    idx, w, _ = orr.forward(gate, x[None], b)
    assert list(idx[0]) == [6, 2]
    s = lambda t: 1 / (1 + math.exp(-t))
    assert w[0] == pytest.approx([2.5 * 0.5 / (0.5 + s(1.5)), 2.5 * s(1.5) / (0.5 + s(1.5))])
    # barred experts leave slots empty; a masked token chooses nothing
    y = np.full((2, 8), -math.inf)
    y[:, 5] = 1.0
    idx, w, load = orr.forward(gate, y, None, [1, 0])
    assert idx.tolist() == [[5, -1], [-1, -1]] and w.tolist() == [[2.5, 0], [0, 0]] and load[5] == 1


def test_adamw_against_its_first_step():
    # at t = 1 from zero moments, m / (1 - b1) = g and v / (1 - b2) = g^2: the step is lr g / (|g| + eps)
    g = np.array([0.3, -2.0, 1e-3])
    p, m, v = oo.step(np.ones(3), g, np.zeros(3), np.zeros(3), 0.1, 0.9, 0.999, 1e-8, 0.5, 1)
    assert p == pytest.approx(1 - 0.05 - 0.1 * g / (np.abs(g) + 1e-8))
    # clipping by the norm scales the gradient only
    q, m2, _ = oo.step(np.ones(3), g, np.zeros(3), np.zeros(3), 0.1, 0.9, 0.999, 1e-8, 0.5, 1, 4.0, 1.0)
    assert m2 == pytest.approx(m / 4)
    a = oo.step32(np.ones(3), g, np.zeros(3), np.zeros(3), 0.1, 0.9, 0.999, 1e-8, 0.5, 1, 16.0, 1.0)
    assert a[0] == pytest.approx(q, rel=1e-6)


def test_e4m3_runs():
    v = oo.e4m3_values()
    assert v[0x7E] == 448 and v[1] == 2.0 ** -9 and v[0x38] == 1 and math.isnan(v[0x7F])
    rng = np.random.default_rng(2)
    x = (rng.standard_normal(77) * np.exp(3 * rng.standard_normal(77))).astype(np.float32)
    x[5] = 0
    for u, positive in ((np.zeros(77), False), (np.full(77, 65535), False), (np.zeros(77), True)):
        y = np.abs(x) if positive else x
        c, s = oo.encode(y, u, positive)
        d = oo.decode(c, s)
        top = np.repeat([np.abs(y[i:i + 32]).max() for i in (0, 32, 64)], 32)[:77]
        # within one step of the value: 2^-3 of it, or of the smallest normal of its run's scale
        # (448 2^e < 2 top, so 2^-6 2^e < top / 14336)
        assert (np.abs(d - y) <= np.maximum(np.abs(y) / 8, top / 14336 / 8)).all()
        if positive:
            assert ((d > 0) == (y > 0)).all()
    # codes that are values already stay what they are, whatever the random bits
    w = v[:127].astype(np.float32)
    c, s = oo.encode(np.concatenate([w, [0]]), np.full(128, 65535), False)
    assert np.array_equal(oo.decode(c, s)[:127], v[:127])
    # the scale is the smallest that holds the largest value: 448 fits its own, the next float not
    assert oo.encode([448.0], [0], False)[1][0] == 127
    assert oo.encode([np.nextafter(np.float32(448), np.float32(500))], [0], False)[1][0] == 128
    assert oo.encode([0.0], [0], False)[1][0] == 0 and oo.encode([math.inf, 1], [0, 0], False)[1][0] == 255


def test_random_bits_are_even_and_rounding_is_unbiased():
    n = 1 << 16
    b = oo.bits(7, 3, n)
    assert len(np.unique(b)) == n                       # one to one within a tensor
    for k in range(32):                                 # each bit set in half of them: 5 sigma = 0.0098
        assert abs(((b >> k) & 1).mean() - 0.5) < 0.0098
    # halves are uncorrelated: 5 / sqrt(n) = 0.0195
    lo, hi = (b & 0xFFFF).astype(float), (b >> 16).astype(float)
    assert abs(np.corrcoef(lo, hi)[0, 1]) < 0.0195
    assert abs(np.corrcoef(lo[1:], lo[:-1])[0, 1]) < 0.0195
    other = (oo.bits(8, 3, n) & 0xFFFF).astype(float)
    assert abs(np.corrcoef(lo, other)[0, 1]) < 0.0195
    # 1.01 lies 8 % of a step above 1.0 (step 1/8): the mean comes back to 5 sigma of its error,
    # 0.125 sqrt(.08 .92 / n) = 1.3e-4
    x = np.full(1024, 1.01, np.float32)
    x[0::32] = 448
    c, s = oo.encode(x, b[:1024] & 0xFFFF, False)
    d = oo.decode(c, s)[np.arange(1024) % 32 != 0]
    assert abs(d.mean() - 1.01) < 5 * 0.125 * math.sqrt(0.08 * 0.92 / len(d))
