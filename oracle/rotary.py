"""Head norms and rotary positions (include/kvq.h) in float64 numpy.  Test
infrastructure."""
from __future__ import annotations

import numpy as np


def turn(x, positions, inv_freq, pair_axis=None, weight=None, eps=0.0, interleaved=False, scale=1.0):
    """x [T, heads, D] -> float64 [T, heads, D].  positions: integers [T] or
    [axes, T] (None: no rotation), inv_freq float32 [pairs]."""
    y = np.asarray(x, np.float64).copy()
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    if positions is None:
        return y
    positions = np.atleast_2d(np.asarray(positions))
    pairs = len(inv_freq)
    axis = np.zeros(pairs, int) if pair_axis is None else np.asarray(pair_axis)
    out = y.copy()
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        # reduced by whole turns in extended precision, as far positions need
        angle = positions[axis[i]].astype(np.longdouble) * np.longdouble(np.float64(inv_freq[i]))
        c, s = (f(angle).astype(np.float64)[:, None] * scale for f in (np.cos, np.sin))
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def slop(x, weight=None, eps=0.0, scale=1.0):
    """A bound on the float32 kernel's error per element, [T, heads, 1].

    Of the pair's sum |x_a w_a| + |x_b w_b| (times the norm factor and |scale|):
    sine and cosine are each off by at most 2^-31 turns of angle, 2^-28.3, and by
    their own rounding, at most 2^-22 with the multiplication by scale and
    weight; two products and one sum 2^-23; the norm's sum of squares, at most
    D + 8 roundings deep but of positive terms, 2^-17 (D 256) on the sum and half
    of that on its root, and its reciprocal root 2^-22.  2^-16 covers them all."""
    y = np.abs(np.asarray(x, np.float64))
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.abs(np.asarray(weight, np.float64))
    return 2.0 ** -16 * 2 * y.max(-1, keepdims=True) * max(1.0, abs(scale))
