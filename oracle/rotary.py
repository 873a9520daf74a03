"""fp64 oracle of rotary positions (include/rotary.h), written from the formula."""
from __future__ import annotations

import numpy as np


def rates(dim, base=10000.0, stretch=1.0, low_turns=0.0, high_turns=0.0, original_len=0.0):
    """Radians a position of the dim / 2 pairs."""
    out = []
    for i in range(dim // 2):
        f = base ** (-2.0 * i / dim)
        g = 0.0
        if high_turns:
            turns = original_len * f / (2 * np.pi)
            g = min(max((turns - low_turns) / (high_turns - low_turns), 0.0), 1.0)
        out.append(f * (g + (1.0 - g) / stretch))
    return np.array(out)


def rotate(x, positions, w, interleaved=False, factor=1.0):
    """x [n, heads, D], rows turned by positions [n]."""
    x = np.asarray(x, np.float64)
    h = len(w)
    out = x.copy()
    for r, p in enumerate(positions):
        c, s = np.cos(p * w), np.sin(p * w)
        for i in range(h):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
            u, v = x[r, :, a], x[r, :, b]
            out[r, :, a] = (u * c[i] - v * s[i]) * factor
            out[r, :, b] = (u * s[i] + v * c[i]) * factor
    return out
