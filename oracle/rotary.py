"""Oracle: rotary positions in float64.

Test infrastructure only (see the package docstring).  Pairs of elements are turned by position * frequency; the angle is
reduced with exact rational arithmetic, so that far positions lose nothing [DEF].
"""

import math
from fractions import Fraction

import numpy as np


def turns_ref(position, turns):
    """The fraction of a turn, in [0, 1), of position * turns (a float64): exact, rounded once."""
    x = Fraction(int(position)) * Fraction(float(turns))
    return float(x - math.floor(x))


def rotary_ref(x, positions, turns, offset=0, interleaved=False, magnitude=1.0, inverse=False):
    """x float64 [rows, heads, dim]; turns float64 [pairs]: turns per position."""
    y, n = np.array(x, dtype=np.float64), len(turns)
    for t, pos in enumerate(positions):
        for i in range(n):
            a, b = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + n + i)
            angle = 2.0 * math.pi * turns_ref(pos, turns[i]) * (-1 if inverse else 1)
            c, s = magnitude * math.cos(angle), magnitude * math.sin(angle)
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return y


def frequencies_ref(dim, base=10000.0):
    """Angle per position of each pair, without scaling."""
    return np.array([base ** (-2.0 * i / dim) for i in range(dim // 2)])
