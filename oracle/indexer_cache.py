"""The 8-bit operands of the indexer's logits, in fp64: layer norm and rotation
of keys, rotation and scales of queries.  Test infrastructure."""
from __future__ import annotations

import numpy as np

from . import kv_fp8 as KF
from . import rope as RO


def keys(k, weight, bias, eps: float, positions, cos_sin, layout: str, first: int):
    """k [T, 128] fp64 -> the values that the codes round, [T, 128]."""
    d = k - k.mean(axis=1, keepdims=True)
    y = d / np.sqrt((d * d).mean(axis=1, keepdims=True) + eps) * weight
    if bias is not None:
        y = y + bias
    return RO.rotate(y[:, None], positions, cos_sin, layout, first)[:, 0]


def queries(q, weights, factor: float, positions, cos_sin, layout: str, first: int):
    """q [T, H, 128] fp64 -> (values divided by their head's scale, scales [T, H],
    weights * factor * scale)."""
    y = RO.rotate(q, positions, cos_sin, layout, first)
    amax = np.where(np.isfinite(y), np.abs(y), 0.0).max(axis=2)
    scale = np.vectorize(lambda a: KF.scale_for(a) or 1.0)(amax)
    return y / scale[..., None], scale, weights * factor * scale
