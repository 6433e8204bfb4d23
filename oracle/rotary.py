"""Oracle of rotary positions in float64.  TEST INFRASTRUCTURE ONLY (see the package header)."""

from __future__ import annotations

import math

import numpy as np


def rotary_frequencies(rot, base=10000.0, factor=1.0, original_len=0.0, low=1.0, high=32.0):
    """Radians a position of each pair."""
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        keep = 0.0
        if original_len > 0:
            keep = min(1.0, max(0.0, (original_len * f / (2 * math.pi) - low) / (high - low)))
        out.append(f * (keep + (1 - keep) / factor))
    return out


def rotary_angles(positions, turns):
    """Angles [T, pairs] from a table of turns times 2^64, reduced by integers."""
    out = np.zeros((len(positions), len(turns)))
    for t, p in enumerate(positions):
        for i, f in enumerate(turns):
            phase = int(p) * int(f) % 2 ** 64
            out[t, i] = 2 * math.pi * ((phase - 2 ** 64 if phase >= 2 ** 63 else phase) / 2 ** 64)
    return out


def rotary(x, angles, interleaved=False, inverse=False, amplitude=1.0):
    """x [T, heads, d] -> (y, mass), mass = A (|x_a| + |x_b|) of the rotated columns."""
    x = np.asarray(x, np.float64)
    y, mass = x.copy(), np.zeros_like(x)
    n = angles.shape[1]
    c, s = np.cos(angles)[:, None], np.sin(angles)[:, None] * (-1 if inverse else 1)
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    y[..., a] = amplitude * (x[..., a] * c - x[..., b] * s)
    y[..., b] = amplitude * (x[..., b] * c + x[..., a] * s)
    for cols in (a, b):
        mass[..., cols] = abs(amplitude) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, mass
