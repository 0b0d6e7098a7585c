"""f / 2 pi in exact arithmetic, and angles from frequencies (not from a plan's rounded table). Test infrastructure."""
import math
from fractions import Fraction

import numpy as np

BITS = 1400


def _arctan_of_inverse(n):
    """2^BITS arctan(1 / n), by its series."""
    term = (1 << BITS) // n
    total, k, sign = term, 1, -1
    while term:
        term //= n * n
        k += 2
        total += sign * (term // k)
        sign = -sign
    return total


TWO_PI = Fraction(8 * (4 * _arctan_of_inverse(5) - _arctan_of_inverse(239)), 1 << BITS)  # Machin


def turns(f):
    """f / 2 pi mod 1 in units of 2^-64, a fraction in [0, 2^64)."""
    return Fraction(f) / TWO_PI % 1 * (1 << 64)


def angles(positions, frequencies):
    """p f mod 2 pi of each position and pair."""
    per = [Fraction(f) / TWO_PI for f in frequencies]
    return 2 * math.pi * np.array([[float(int(p) * t % 1) for t in per] for p in positions])
