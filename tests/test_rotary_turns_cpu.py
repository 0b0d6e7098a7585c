"""lin_rotary_turns against f / 2 pi in exact arithmetic: 0.6 of a unit of 2^-64 (half a unit for the rounding; the
quotient itself is good to 2^-105 of its size, 2^-68 for frequencies below 2^40)."""
import ctypes
import math
import random
from fractions import Fraction

import serving_turns as exact
import transformer_linear_layer_gb300 as tll


def turns(values):
    out = (ctypes.c_ulonglong * len(values))()
    assert tll.library().lin_rotary_turns((ctypes.c_double * len(values))(*values), len(values), out) == tll.OK
    return list(out)


def test_all_64_bits_are_right():
    assert abs(float(exact.TWO_PI) - 2 * math.pi) == 0
    rng = random.Random(5)
    values = [0.0, -0.0, 1.0, -1.0, 0.5, 1e-9, -1e-9, 1e-18, -1e-18, 2.0 ** -60, 2.0 ** -66, -2.0 ** -66, 5e-324, 500.25, 2 * math.pi,
              -2 * math.pi, math.pi, 2.0 ** 39 + 0.5, 2.0 ** 40, -2.0 ** 40]
    values += [10000.0 ** (-2 * i / 128) for i in range(64)] + [500000.0 ** (-2 * i / 64) / 16 for i in range(32)]
    values += [rng.choice((-1, 1)) * 2.0 ** rng.uniform(-70, 40) for _ in range(3000)]
    for f, got in zip(values, turns(values)):
        off = (got - exact.turns(f)) % (1 << 64)
        off = min(off, (1 << 64) - off)
        assert off <= Fraction(6, 10), (f, float(off))


def test_far_frequencies_are_taken():
    """Larger ones lose digits (2^-104 of the quotient), and none leaves the range of the arithmetic."""
    values = [s * 2.0 ** e * 1.37 for e in (41, 52, 53, 63, 64, 80, 103, 104, 200, 1022) for s in (1, -1)]
    for f, got in zip(values, turns(values)):
        off = (got - exact.turns(f)) % (1 << 64)
        off = min(off, (1 << 64) - off)
        assert off <= 1 + Fraction(abs(f)) / 6 / (1 << 40), (f, float(off))


def test_angles_follow_the_frequencies_at_far_positions():
    """A plan's table against its frequencies, not against itself: |p| 2^-62 radians."""
    r = tll.Rotary(64, base=500000.0, scaling="yarn", factor=4.0, original_length=2048, device="cpu")
    places = [1, 10 ** 6, -(10 ** 6), 2 ** 31 - 1, 2 ** 50, -(2 ** 50) - 1, 2 ** 62 + 12345]
    want = exact.angles(places, r.frequencies)
    for i, p in enumerate(places):
        for j, t in enumerate(r.turns.tolist()):
            got = p * t % (1 << 64) / 2.0 ** 64 * 2 * math.pi
            off = abs(got - want[i, j])
            assert min(off, 2 * math.pi - off) <= abs(p) * 2.0 ** -62 + 2.0 ** -48
