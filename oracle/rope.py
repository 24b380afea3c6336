"""f64 reference for rotary positions (test infrastructure only)."""

import math
from fractions import Fraction

import numpy as np

#: pi to 60 digits.
PI = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)


def angle(position, frequency):
    """position * frequency modulo a turn, in -pi .. pi, from exact arithmetic."""
    turns = Fraction(int(position)) * Fraction(float(frequency)) / (2 * PI)
    left = turns - math.floor(turns + Fraction(1, 2))
    return float(left * 2 * PI)


def rotate(x, positions, frequencies, interleaved=False, amplitude=1.0, inverse=False):
    """f64 rows x [rows, heads, dim], the first 2 * len(frequencies) channels of each head turned."""
    x = np.asarray(x, np.float64)
    out = x.copy()
    half = len(frequencies)
    for t, p in enumerate(positions):
        for i, f in enumerate(frequencies):
            a = angle(p, f) * (-1 if inverse else 1)
            c, s = amplitude * math.cos(a), amplitude * math.sin(a)
            m, n = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            out[t, :, m] = c * x[t, :, m] - s * x[t, :, n]
            out[t, :, n] = s * x[t, :, m] + c * x[t, :, n]
    return out
