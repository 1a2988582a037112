"""The oracle's stochastic rounding to E4M3 against rational arithmetic."""
import math
from fractions import Fraction

import numpy as np

from oracle import optim as oo


def by_definition(x, e, u, positive):
    """Signed value of one rounded element under the scale 2^e."""
    a = Fraction(abs(float(x))) / Fraction(2) ** e
    step = Fraction(1, 512)
    while a >= 16 * step:
        step *= 2
    k = math.floor(a / step + Fraction(int(u), 65536))
    if positive and a > 0:
        k = max(k, 1)
    return (-1 if x < 0 else 1) * k * step * Fraction(2) ** e


def test_codes_are_the_definitions():
    rng = np.random.default_rng(4)
    x = (rng.standard_normal(2048) * np.exp(4 * rng.standard_normal(2048))).astype(np.float32)
    u = rng.integers(0, 65536, 2048)
    for positive in (False, True):
        y = np.abs(x) if positive else x
        c, s = oo.encode(y, u, positive)
        d = oo.decode(c, s)
        assert all(d[j] == by_definition(y[j], int(s[j // 32]) - 127, u[j], positive) for j in range(2048))


def test_a_value_short_of_its_border_stays_below():
    """Border a = i - u / 2^16 steps: there the code is i, one fp32 unit below it is i - 1, also where the unit
    is so small that a sum in fp32 loses it (a below half a step)."""
    rng = np.random.default_rng(5)
    x, u, want = [], [], []
    for r in range(64):
        i = rng.integers(1, 9, 31)
        b = rng.integers(0, 65536, 31)
        b[:8], i[:8] = 65536 - (1 << np.arange(8)), 1
        a = ((i * 65536 - b) / 65536 * 2.0 ** -9).astype(np.float32)
        low = rng.random(31) < 0.5
        x.append(np.concatenate([[448.0], np.where(low, np.nextafter(a, np.float32(0)), a)]))
        u.append(np.concatenate([[0], b]))
        want.append(np.concatenate([[0x7E], i - low]))
    c, s = oo.encode(np.concatenate(x), np.concatenate(u), False)
    assert (s == 127).all() and np.array_equal(c, np.concatenate(want))
