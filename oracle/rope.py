"""Rotary positions in extended precision: the rotation of each pair of a
head's elements by position times frequency."""

import numpy as np


def rotate(x, positions, inv_freq, interleaved: bool = False, scale: float = 1.0,
           inverse: bool = False):
    """x [rows, heads, dim] (fp64), positions [rows], inv_freq [n]: the first
    2 n elements of each head turned, the others as they are.  Rows whose
    position is None are as they are."""
    x = np.asarray(x, np.float64)
    f = np.asarray(inv_freq, np.longdouble)
    n = len(f)
    out = x.copy()
    for i, p in enumerate(positions):
        if p is None:
            continue
        a = (-1 if inverse else 1) * np.longdouble(int(p)) * f
        c, s = np.cos(a).astype(np.float64) * scale, np.sin(a).astype(np.float64) * scale
        first = np.arange(n) * 2 if interleaved else np.arange(n)
        second = first + (1 if interleaved else n)
        u, v = x[i][:, first], x[i][:, second]
        out[i][:, first] = u * c - v * s
        out[i][:, second] = v * c + u * s
    return out


def packed_positions(rows: int, cu):
    """Position of each row of a packed batch; None past the last offset."""
    pos = [None] * rows
    for a, b in zip(cu[:-1], cu[1:]):
        for r in range(a, b):
            pos[r] = r - a
    return pos
