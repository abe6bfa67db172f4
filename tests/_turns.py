"""Angles as exact fractions of a turn, with pi from J. Machin's formula in integers."""
from fractions import Fraction

import numpy as np

BITS = 400


def _arctan_inverse(x, one):
    total, term, n, sign = 0, one // x, 1, 1
    while term:
        total += sign * (term // n)
        term //= x * x
        n, sign = n + 2, -sign
    return total


_ONE = 1 << (BITS + 32)
PI = Fraction(4 * (4 * _arctan_inverse(5, _ONE) - _arctan_inverse(239, _ONE)), _ONE)  # to 2^-400


def turns(freq, position=1):
    """position x freq (radians, a double as it is) as a fraction of a turn in [0, 1)."""
    return (Fraction(float(freq)) * int(position) / (2 * PI)) % 1


def cos_sin(positions, inv_freq):
    """positions [N][pairs] int, inv_freq [pairs]: cos and sin, float64."""
    c, s = np.zeros(positions.shape), np.zeros(positions.shape)
    for n, i in np.ndindex(*positions.shape):
        t = turns(inv_freq[i], positions[n, i])
        quarter = int(t * 4 + Fraction(1, 2))
        rest = float(t - Fraction(quarter, 4)) * 2 * np.pi  # at most an eighth of a turn: to 2^-53
        a, b = np.cos(rest), np.sin(rest)
        for _ in range(quarter % 4):
            a, b = -b, a
        c[n, i], s[n, i] = a, b
    return c, s
