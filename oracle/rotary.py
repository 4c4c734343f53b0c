"""Plain statement of the rotary positions and the heads' norms in numpy.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  Angles are worked out
in 80 bits (the position times the frequency, less whole turns), all else in 64.
"""
from __future__ import annotations

import math

import numpy as np

HALVES, PAIRS = range(2)
TURN = np.longdouble("6.283185307179586476925286766559")


def frequencies(dims, base, scaling="plain", factor=1.0, original=0.0, low=0.0, high=0.0):
    """Radians a token of each pair, by the definitions of include/nf4.h."""
    if scaling == "base" and dims > 2:
        base *= factor ** (dims / (dims - 2))
    out = []
    for i in range(dims // 2):
        f = base ** (-2 * i / dims)
        if scaling == "linear":
            f /= factor
        elif scaling == "smooth":
            turns = original * f / (2 * math.pi)
            r = 1 - (turns - low) / (high - low)
            r = min(max(r, 0.0), 1.0)
            f = f * (1 - r) + f / factor * r
        elif scaling == "ramp":
            def number(turns):
                return dims * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))
            a, b = max(math.floor(number(high)), 0), min(math.ceil(number(low)), dims - 1)
            r = (i - a) / ((b if b != a else a + 0.001) - a)
            r = min(max(r, 0.0), 1.0)
            f = f * (1 - r) + f / factor * r
        out.append(f)
    return np.array(out)


def norm(x, weight, eps):
    """x [..][D] in 64 bits."""
    with np.errstate(all="ignore"):
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps))) * weight


def pair_indexes(dims, layout):
    if layout == HALVES:
        return np.arange(dims // 2), np.arange(dims // 2) + dims // 2
    return np.arange(0, dims, 2), np.arange(1, dims, 2)


def rotate(x, positions, frequency, layout, gain=1.0):
    """x: float64 [rows][heads][D].  Returns the result and, for error bounds,
    the magnitude |a| + |b| of each value's pair (0 where nothing turns)."""
    dims = 2 * len(frequency)
    y, mag = x.copy(), np.zeros_like(x)
    a, b = pair_indexes(dims, layout)
    angle = np.asarray(positions, np.longdouble)[:, None] * np.asarray(frequency, np.longdouble)
    angle = (angle - np.rint(angle / TURN) * TURN).astype(np.float64)[:, None, :]
    c, s = np.cos(angle) * gain, np.sin(angle) * gain
    with np.errstate(all="ignore"):
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
        mag[..., a] = mag[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(gain)
    return y, mag
