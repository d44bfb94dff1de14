"""Phases of the rotary positions against 60-digit arithmetic (no GPU): 64 bits of the frequencies
given, so that far positions have the angle p * f."""
import math
from fractions import Fraction

import numpy as np
import pytest

import context_parallelism_gb300 as up
from oracle import rope_ref

PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


def _off(word, f):
    """Units of 2^-64 of a turn between a phase and the frequency."""
    d = (word - Fraction(f) / (2 * PI) * 2 ** 64) % 2 ** 64
    return min(d, 2 ** 64 - d)


def _frequencies():
    f = [1.0, 0.5, 3.0, 100.0, 1e-3, 1e-6, 1e-12, 1e-19, 2.0 ** -70, 0.0, math.pi, 2 * math.pi,
         math.nextafter(2 * math.pi, 0), math.nextafter(2 * math.pi, 7), 7 * math.pi, 12345.678,
         1e9, 2.0 ** 40 - 0.5]
    for kw in (dict(theta=500000.0), dict(scaling=up.UPIPE_ROPE_LINEAR, factor=8.0),
               dict(scaling=up.UPIPE_ROPE_NTK, factor=8.0),
               dict(scaling=up.UPIPE_ROPE_BY_PARTS, factor=8.0, trained_len=8192)):
        f += up.upipe_rope_frequencies(128, **kw)[0]
    rng = np.random.default_rng(1)
    f += list(np.exp(rng.uniform(-40, 25, 500)))
    return f + [-x for x in f]


def test_phases_are_the_frequencies_to_half_a_unit():
    """Rounded to nearest: half a unit and the quarter that the quotient may be off by."""
    f = [float(x) for x in _frequencies()]
    for x, w in zip(f, up.upipe_rope_phases(f)):
        assert 0 <= w < 2 ** 64 and _off(w, x) <= Fraction(3, 4), (x, w)


@pytest.mark.parametrize("pos", [1 << 24, (1 << 31) + 1, 10 ** 12, -(1 << 40)])
def test_far_positions_have_the_angle_of_the_frequency(pos):
    """|p| 3/4 units of 2^-64 of a turn at the most, whatever the frequency's size."""
    f, _ = up.upipe_rope_frequencies(64, theta=500000.0)
    w = up.upipe_rope_phases(f)
    x = np.zeros((1, 1, 64))
    x[..., :32] = 1.0
    y = rope_ref(x, [pos], w)[0, 0]
    for i in range(32):
        turns = (pos * Fraction(f[i]) / (2 * PI)) % 1
        a = 2 * math.pi * float(turns)
        tol = 2 * math.pi * 0.75 * abs(pos) * 2.0 ** -64 + 1e-14
        assert abs(y[i] - math.cos(a)) <= tol and abs(y[32 + i] - math.sin(a)) <= tol
