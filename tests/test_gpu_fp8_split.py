"""GPU parity of dsa_sparse_mla_decode_fp8 on both sides of the numbers of
(row, head group) pairs that are split over eight, four and two CTAs, against the
fp64 softmax, with the bounds of tests/test_gpu_fp8_mixed_scales.py."""
import numpy as np
import pytest

from tests.test_gpu_fp8_mixed_scales import _codes, _compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,H", [(7, 128), (8, 128), (9, 128), (15, 64), (16, 48), (18, 128), (19, 128),
                                    (36, 64), (37, 20), (38, 128), (39, 128), (76, 64), (77, 64)])
@pytest.mark.parametrize("K", [2048, 1100])
def test_every_number_of_parts(rows, H, K):
    rng = np.random.default_rng(rows)
    n, block = 4096, 64
    scales = np.exp2(rng.integers(-8, -4, n // block)).astype(np.float64)
    q = rng.standard_normal(576) * 2.0
    _compare(rows, H, q, _codes(rng, n), scales, block, rng.permutation(n)[:K])
