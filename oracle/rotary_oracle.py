"""Plain fp64 oracle of rotary positions: test infrastructure only."""
from __future__ import annotations

import numpy as np


def frequencies(rotary_dim, base=10000.0):
    """Radians per position of each pair: base^(-2 i / rotary_dim)."""
    return np.array([float(base) ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)])


def pairs(rotary_dim, adjacent):
    """The two columns of every pair."""
    i = np.arange(rotary_dim // 2)
    return (2 * i, 2 * i + 1) if adjacent else (i, i + rotary_dim // 2)


def rotate(x, positions, freq, axis=None, adjacent=False, scale=1.0, inverse=False):
    """x [..., heads, dim] by positions [axes, ...] -> (y, size): size bounds what a rounding of a cosine
    or of a product can move y by, |x_a| + |x_b| of its pair."""
    x, positions = np.asarray(x, np.float64), np.asarray(positions, np.float64)
    axis = np.zeros(len(freq), int) if axis is None else np.asarray(axis)
    y, size = x.copy(), np.zeros_like(x)
    a, b = pairs(2 * len(freq), adjacent)
    for i, f in enumerate(freq):
        w = (positions[axis[i]] * f)[..., None] * (-1 if inverse else 1)
        xa, xb = x[..., a[i]], x[..., b[i]]
        y[..., a[i]] = (xa * np.cos(w) - xb * np.sin(w)) * scale
        y[..., b[i]] = (xb * np.cos(w) + xa * np.sin(w)) * scale
        size[..., a[i]] = size[..., b[i]] = (np.abs(xa) + np.abs(xb)) * abs(scale)
    return y, size
