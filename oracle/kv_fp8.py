"""The 8-bit MLA cache: e4m3 codes, a power-of-two scale for each block of
slots, and the insert of new rows.  Test infrastructure.

e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits, subnormals in steps of
2^-9, largest value 448, code 0x7F the NaN; no infinity.
"""
from __future__ import annotations

import numpy as np

MAX = 448.0


def decode(codes) -> np.ndarray:
    """fp64 values of e4m3 codes."""
    c = np.asarray(codes, np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e > 0, (1.0 + m / 8.0) * 2.0 ** (e - 7.0), m * 2.0 ** -9)
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


_FINITE = decode(np.arange(0x7F, dtype=np.uint8))     # ascending, codes 0 .. 0x7E


def encode(x) -> np.ndarray:
    """Nearest e4m3 code (ties to the even code), saturating at +-448; NaN to
    the NaN code."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=np.inf, neginf=-np.inf)), MAX)
    hi = np.clip(np.searchsorted(_FINITE, a, side="left"), 1, len(_FINITE) - 1)
    lo = hi - 1
    up, down = _FINITE[hi] - a, a - _FINITE[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def scale_for(amax: float) -> float:
    """The smallest power of two s >= 2^-126 with amax <= 448 s (0 for 0)."""
    if amax == 0.0:
        return 0.0
    s = 2.0 ** -126
    while amax > MAX * s:
        s *= 2.0
    return s


def insert(cache, scales, rows, slots):
    """(codes, scales) after the rows [T, 576] (fp64 values of bf16) went to
    their slots, block by block."""
    cache, scales = np.array(cache), np.array(scales, np.float32)
    block = cache.shape[0] // scales.shape[0]
    last = {int(s): t for t, s in enumerate(slots) if 0 <= s < cache.shape[0]}
    for b in sorted({s // block for s in last}):
        mine = {s: t for s, t in last.items() if s // block == b}
        new = np.array([rows[t] for t in mine.values()])
        old = float(scales[b]) if scales[b] > 0 else 0.0
        scale = max(old, scale_for(float(np.where(np.isfinite(new), np.abs(new), 0.0).max())))
        scales[b] = scale
        div = np.float32(scale if scale > 0 else 1.0)
        if old > 0 and scale > old:
            ratio = np.float32(old) / div
            for s in range(b * block, (b + 1) * block):
                if s not in mine:
                    cache[s] = encode((decode(cache[s]).astype(np.float32) * ratio))
        with np.errstate(invalid="ignore", over="ignore"):
            for s, t in mine.items():
                cache[s] = encode(np.asarray(rows[t], np.float32) / div)
    return cache, scales


def values(cache, scales) -> np.ndarray:
    """fp64 values of the whole cache."""
    block = cache.shape[-2] // scales.shape[-1]
    return decode(cache) * np.repeat(np.asarray(scales, np.float64), block, axis=-1)[..., None]
