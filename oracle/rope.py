"""Rotation tables (scaled for long contexts) and rotary positions, in fp64.
Test infrastructure.

The frequencies are the published definitions: w_i = base^(-2i/d); linear
position interpolation divides them by the factor; the NTK-aware variant raises
the base by factor^(d/(d-2)); YaRN ("YaRN: Efficient Context Window Extension
of Large Language Models") interpolates the pairs that turn slowly within the
trained context, with a linear ramp over pair indices as the released models
take it.
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(rot_dim: int, base: float, scaling=None, factor: float = 1.0,
                orig_max_pos: int = 4096, beta_fast: float = 32.0,
                beta_slow: float = 1.0) -> np.ndarray:
    """Angle per position of each of the rot_dim / 2 pairs, fp64."""
    d = float(rot_dim)
    if scaling == "ntk" and rot_dim > 2:
        base = base * factor ** (d / (d - 2.0))
    w = np.array([base ** (-2.0 * i / d) for i in range(rot_dim // 2)])
    if scaling == "linear":
        return w / factor
    if scaling != "yarn":
        return w
    index = lambda turns: (d * math.log(orig_max_pos / (2 * math.pi * turns))   # noqa: E731
                           / (2 * math.log(base)))
    low = max(math.floor(index(beta_fast)), 0)
    high = min(math.ceil(index(beta_slow)), d - 1)
    ramp = np.clip((np.arange(rot_dim // 2) - low) / max(high - low, 0.001), 0.0, 1.0)
    return w * (1.0 - ramp) + w / factor * ramp


def table(max_pos: int, rot_dim: int, base: float, amplitude: float = 1.0, **scaling):
    """[max_pos, rot_dim] fp64: cosines, then sines."""
    a = np.arange(max_pos, dtype=np.float64)[:, None] * frequencies(rot_dim, base, **scaling)
    return amplitude * np.concatenate([np.cos(a), np.sin(a)], axis=1)


def rotate(x, positions, cos_sin, layout: str, first: int = 0, inverse: bool = False):
    """x [T, H, D] fp64 with [first, first + rot_dim) of every head turned by
    cos_sin [max_pos, rot_dim] at positions [T]; a position outside the table
    leaves its token as it is."""
    x = np.array(x, np.float64)
    n = cos_sin.shape[1]
    for t, p in enumerate(np.asarray(positions)):
        if not 0 <= p < cos_sin.shape[0]:
            continue
        c = np.asarray(cos_sin[p, :n // 2], np.float64)
        s = np.asarray(cos_sin[p, n // 2:], np.float64) * (-1.0 if inverse else 1.0)
        r = x[t, :, first:first + n]
        ia, ib = ((slice(0, n, 2), slice(1, n, 2)) if layout == "interleaved"
                  else (slice(0, n // 2), slice(n // 2, n)))
        a, b = r[:, ia].copy(), r[:, ib].copy()
        r[:, ia] = a * c - b * s
        r[:, ib] = b * c + a * s
    return x
