"""Rotary embedding with one position per axis — test infrastructure only.

The rotary reading of ``oracle.rope`` (pair i turned by position x theta_i), with the
D/2 feature pairs cut into one run per axis: pair i of axis a is turned by
positions[a] x theta_i. ``freqs`` "shared": theta_i = base^(-2i/D) over all pairs;
"per_axis": theta = base^(-j/n), j the pair's index within the axis's n pairs.
``pairing`` "adjacent": pair i is features (2i, 2i + 1); "half": (i, i + D/2). All
arithmetic float64.
"""
from __future__ import annotations

import numpy as np


def angles(positions, sections, D: int, base: float = 10000.0, freqs: str = "shared"):
    """positions [axes, ...] -> turning angle of each pair [..., D/2]."""
    out = []
    i = 0
    for a, n in enumerate(sections):
        for j in range(n):
            theta = base ** (-j / n) if freqs == "per_axis" else base ** (-2.0 * i / D)
            out.append(np.asarray(positions[a], np.float64) * theta)
            i += 1
    assert i == D // 2
    return np.stack(out, axis=-1)


def rotate(x, angle, pairing: str = "adjacent", inverse: bool = False):
    """x [..., H, D] turned by angle [..., D/2] (the same for every head)."""
    x = np.asarray(x, np.float64)
    D = x.shape[-1]
    c, s = np.cos(angle)[..., None, :], np.sin(angle)[..., None, :]
    if inverse:
        s = -s
    out = np.empty_like(x)
    even, odd = (slice(0, None, 2), slice(1, None, 2)) if pairing == "adjacent" else (slice(0, D // 2), slice(D // 2, None))
    out[..., even] = x[..., even] * c - x[..., odd] * s
    out[..., odd] = x[..., even] * s + x[..., odd] * c
    return out
