"""Norm and rotation of query and key heads in float64 (no counterpart in the reference).

    y = x / sqrt(mean(x^2) + eps) * (weight + offset)
    pair i of the first 2 * len(inv_freq) dims turns by position[axis(i)] * inv_freq[i]
"""

from __future__ import annotations

import numpy as np


def axis_of(i, sections, cycle):
    """The axis of frequency i: blocks of `sections` frequencies, or the axes in turn while each has
    some left (then axis 0)."""
    if cycle:
        a = i % len(sections)
        return a if i // len(sections) < sections[a] else 0
    return int(np.searchsorted(np.cumsum(sections), i, side="right"))


def norm_rotate(x, positions, inv_freq, weight=None, eps=1e-6, offset=0.0, sections=None, cycle=False, adjacent=False,
                amplitude=1.0):
    """x [T, H, D], positions [T] or [axes, T]; returns float64 [T, H, D] and the magnitude of what each
    value was made of (its pair's, or its own)."""
    x = np.asarray(x, dtype=np.float64)
    pos = np.atleast_2d(np.asarray(positions, dtype=np.float64))
    freq = np.asarray(inv_freq, dtype=np.float64)
    half = len(freq)
    sections = [half] if sections is None else list(sections)
    y = x
    if weight is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (np.asarray(weight, dtype=np.float64) + offset)
    angle = np.stack([pos[axis_of(i, sections, cycle)] * freq[i] for i in range(half)], -1)[:, None]  # [T, 1, half]
    c, s = amplitude * np.cos(angle), amplitude * np.sin(angle)
    at = (np.arange(half) * 2, np.arange(half) * 2 + 1) if adjacent else (np.arange(half), np.arange(half) + half)
    out, size = y.copy(), np.abs(y)
    a, b = y[..., at[0]], y[..., at[1]]
    out[..., at[0]], out[..., at[1]] = a * c - b * s, b * c + a * s
    size[..., at[0]] = size[..., at[1]] = abs(amplitude) * np.hypot(a, b)
    return out, size
