"""How exact a rotation's angle is at any position: the turns of a frequency in fixed
point, and the oracle's own angle, against rational arithmetic (no GPU needed)."""
import math
from fractions import Fraction

import numpy as np
import pytest

import segment_masked_causal_gb300 as pa
from oracle import rotary

TWO_PI = Fraction("6.283185307179586476925286766559005768394338798750211641949889")


@pytest.fixture(scope="module", autouse=True)
def L():
    from segment_masked_causal_gb300 import build
    build.build()
    return pa.lib()


def off(a, b):
    d = (a - b) % 1
    return min(d, 1 - d)


@pytest.mark.parametrize("theta", [1e4, 5e5, 1.5])
def test_turns_at_the_last_position(theta):
    """Turns to half a step of 2^-64 and the small remainder of two doubles (2^-100 of the turns),
    so a product with any position is within 2^-32 of a turn."""
    r = pa.Rotary(128, theta=theta)
    for f, t in zip(r.frequencies, r.c.turns):
        exact = Fraction(f) / TWO_PI
        assert off(Fraction(t, 1 << 64), exact) <= Fraction(1, 1 << 64)
        assert off(Fraction(t, 1 << 64) * (2 ** 31 - 1), exact * (2 ** 31 - 1)) <= Fraction(1, 1 << 33)


def test_turns_of_any_frequency():
    given = [0.0, -0.0, 1.0, -1.0, 1e-3, -1e-9, 1e-30, 2 * math.pi, -math.pi, math.pi, 7.5, 1e3 + 0.1, -12345.678, 2.0 ** 40 + 0.5,
             -3.0e10, 5e-324]
    r = pa.Rotary(32, frequencies=given)
    for f, t in zip(given, r.c.turns):
        assert off(Fraction(t, 1 << 64), Fraction(f) / TWO_PI) <= Fraction(1, 1 << 64) + abs(Fraction(f)) / (1 << 104)
    huge = pa.Rotary(16, frequencies=[2.0 ** 60, 1e18, 1e100, 1e308, -1e308, 2.0 ** 52, 2.0 ** 53 * math.pi, -2.0 ** 63])
    assert len(huge.c.turns) == 64  # taken as they are: finite is all that is asked


@pytest.mark.parametrize("pos", [1, 12345, 2 ** 20 + 3, 2 ** 31 - 1, -2 ** 31])
def test_oracle_drops_whole_turns(pos):
    f = rotary.frequencies(128, theta=5e5)
    x = np.zeros(128)
    x[:64] = 1
    y = rotary.rotate(x, np.array(pos), f)
    for i in range(64):
        part = Fraction(f[i]) * pos / TWO_PI % 1
        a = float(part * TWO_PI)
        # 2^-64 of the angle in long double, 2^-63 of 2 pi for each whole turn, and the last roundings
        assert abs(y[i] - math.cos(a)) <= 1e-9 and abs(y[i + 64] - math.sin(a)) <= 1e-9
