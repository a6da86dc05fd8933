"""Rotation tables at far positions, against the definition in 80-digit decimal
arithmetic (tests/test_rope_steps.py).

Tolerance, from the arithmetic, in units of 2^-24 of the amplitude.  The angle is
cut to 2^-32 turns (2 pi 2^-32: 0.03), and its step is off by 2^-65 turns, 2^-37 turns
at position 2^28 (0.001).  Within an eighth of a turn x = u (2 pi 2^-32) has three
roundings, of the integer, the constant and the product: 3 |x|, which moves the
sine by 3 x cos x and the cosine by 3 x sin x, at most 1.7 at x = pi / 4.  The
series ends below 2^-29 (0.03).  Evaluating it: of the sine's x^3 t, at most 0.08
with four roundings, 0.4; of the cosine's x^2 t, at most 0.31 with two, 0.7; and the
last sum's rounding, 0.5.  The product with the amplitude: 1.  Below 4 in all:
2.4e-7 of the amplitude."""
import math

import numpy as np
import pytest
import torch

from tests.test_rope_steps import NONE, NTK, YARN, _exact

pytestmark = pytest.mark.gpu

KINDS = {NONE: None, NTK: "ntk", YARN: "yarn"}


@pytest.mark.parametrize("max_pos,rot,base,kind,factor,orig", [
    (2 ** 28, 4, 1e4, NONE, 1.0, 4096), (2 ** 28 - 5, 2, 1e4, NONE, 1.0, 4096),
    (2 ** 26, 12, 5e5, NTK, 8.0, 4096), (2 ** 27, 6, 1e4, YARN, 32.0, 8192)])
def test_far_positions_are_as_exact_as_near_ones(max_pos, rot, base, kind, factor, orig):
    import dsa_sparse_indexer_gb300 as dsa
    table = dsa.rope_table(max_pos, rot, base, KINDS[kind], factor, orig, amplitude=1.25)
    steps = _exact(rot, base, kind, factor, orig, 32.0, 1.0)
    positions = sorted({0, 1, 2, max_pos - 1, *(max_pos - 1 - k * 131 for k in range(500)),
                        *(max_pos * k // 500 for k in range(500))})
    got = table[torch.tensor(positions, device="cuda")].double().cpu().numpy()
    for row, p in zip(got, positions):
        turns = [float((s * p / 2 ** 64) % 1) for s in steps]
        want = [1.25 * f(2 * math.pi * t) for f in (math.cos, math.sin) for t in turns]
        assert np.abs(row - want).max() <= 1.25 * 4 * 2.0 ** -24, p
