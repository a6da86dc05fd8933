"""Pins of the rotation and 8-bit cache oracles (CPU): hand-worked values,
properties of rotations, the e4m3 grid, the insert against rows put in one at
a time."""
import numpy as np
import pytest
import torch

from oracle import kv_fp8 as KF
from oracle import pcp_prefill as PP
from oracle import rope as RO


def test_frequencies_by_hand():
    np.testing.assert_allclose(RO.frequencies(4, 100.0), [1.0, 0.1])
    np.testing.assert_allclose(RO.frequencies(4, 100.0, "linear", 4.0), [0.25, 0.025])
    # NTK: base 100 * 4^(4/2) = 1600, so the slowest pair is 1600^(-1/2)
    np.testing.assert_allclose(RO.frequencies(4, 100.0, "ntk", 4.0), [1.0, 0.025])
    # YaRN: the fastest pairs as they are, the slowest interpolated
    w = RO.frequencies(64, 10000.0)
    y = RO.frequencies(64, 10000.0, "yarn", 40.0, 4096)
    np.testing.assert_array_equal(y[:11], w[:11])
    np.testing.assert_allclose(y[23:], w[23:] / 40.0, rtol=1e-12)
    assert ((y[11:23] < w[11:23]) & (y[11:23] > w[11:23] / 40.0)).all()


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rotation_keeps_lengths_and_turns_back(layout):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 3, 20))
    cs = RO.table(50, 12, 10000.0)
    pos = np.array([0, 7, 49, 50, -1])
    y = RO.rotate(x, pos, cs, layout, first=3)
    np.testing.assert_allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
    np.testing.assert_array_equal(y[..., :3], x[..., :3])
    np.testing.assert_array_equal(y[3:], x[3:])
    np.testing.assert_allclose(RO.rotate(y, pos, cs, layout, first=3, inverse=True), x, atol=1e-12)


def test_scores_depend_on_the_distance_only():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    cs = RO.table(200, 16, 10000.0)
    at = lambda v, p: RO.rotate(v, [p], cs, "half")[0, 0]     # noqa: E731
    np.testing.assert_allclose(at(q, 30) @ at(k, 10), at(q, 150) @ at(k, 130))


def test_interleaved_is_the_cache_rows_rotation():
    rng = np.random.default_rng(3)
    x, cs = rng.standard_normal((4, 64)), RO.table(9, 64, 10000.0)
    pos = np.array([8, 0, 3, 5])
    want = PP.rope_interleaved(x, cs[pos, :32], cs[pos, 32:])
    np.testing.assert_allclose(RO.rotate(x[:, None], pos, cs, "interleaved")[:, 0], want)


def test_e4m3_grid():
    assert KF.decode([0x00, 0x01, 0x08, 0x38, 0x7E, 0xB8]).tolist() == \
        [0.0, 2.0 ** -9, 2.0 ** -6, 1.0, 448.0, -1.0]
    finite = np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)
    np.testing.assert_array_equal(KF.encode(KF.decode(finite)), finite)
    # ties to the even code, saturation, NaN
    np.testing.assert_array_equal(KF.encode([1.0625, 1.1875, 1000.0, -np.inf, 2.0 ** -10]),
                                  [0x38, 0x3A, 0x7E, 0xFE, 0x00])
    assert KF.encode([np.nan])[0] == 0x7F
    x = np.random.default_rng(4).standard_normal(5000) * 100
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(KF.encode(x), want)


@pytest.mark.parametrize("amax,want", [(0.0, 0.0), (448.0, 1.0), (449.0, 2.0), (3.5, 2.0 ** -7),
                                       (1e-45, 2.0 ** -126), (3.38e38, 2.0 ** 120)])
def test_scale_is_the_smallest_power_of_two(amax, want):
    assert KF.scale_for(amax) == want


def test_insert_together_is_insert_one_by_one_when_scales_hold():
    """Rows of falling magnitude: the first one's scale serves them all."""
    rng = np.random.default_rng(5)
    rows = rng.uniform(-1, 1, (6, 576)) * 2.0 ** -np.arange(6)[:, None]
    rows[0, 0] = 1.0
    slots = [3, 1, 9, 2, 3, -1]
    cache, scales = np.zeros((16, 576), np.uint8), np.zeros(4, np.float32)
    c1, s1 = KF.insert(cache, scales, rows, slots)
    c2, s2 = cache, scales
    for t in range(6):
        c2, s2 = KF.insert(c2, s2, rows[t:t + 1], slots[t:t + 1])
    # slot 3 was named twice: the last token's row
    np.testing.assert_array_equal(c1[3], KF.encode(rows[4] / s1[0]))
    np.testing.assert_array_equal(c1[9], c2[9])
    assert s1[2] == s2[2] > 0 and s1[1] == s1[3] == 0


def test_a_larger_row_moves_the_blocks_codes():
    cache, scales = np.zeros((4, 576), np.uint8), np.zeros(1, np.float32)
    small, large = np.full((1, 576), 3.0), np.full((1, 576), 3.0 * 2 ** 6)
    cache, scales = KF.insert(cache, scales, small, [1])
    assert scales[0] == 2.0 ** -7
    cache, scales = KF.insert(cache, scales, large, [2])
    assert scales[0] == 0.5
    v = KF.values(cache, scales)
    assert (v[1] == 3.0).all() and (v[2] == 192.0).all()
