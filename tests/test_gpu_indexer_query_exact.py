"""dsa_indexer_query_fp8 beside the fp64 oracle (oracle/indexer_cache.py), code by
code and scale by scale.

No tolerance: a code is the exact value's, rounded once.  The oracle's fp64 holds a
turned value to 2^-53 of its larger product (a bf16 value times an fp32 entry is
exact in it), so that it and the exact value round apart only where a value is
nearer than that to a border; the inputs are fixed, and none of them is."""
import numpy as np
import pytest
import torch

from oracle import indexer_cache as IC
from oracle import kv_fp8 as KF
from oracle import rope as RO

pytestmark = pytest.mark.gpu

TURNS = [("half", 64, 0), ("interleaved", 64, 0), ("half", 128, 0), ("interleaved", 2, 126), ("half", 6, 5),
         ("interleaved", 50, 33), ("half", 64, 64)]
INF = float("inf")


def pairs_of(layout, rot, first):
    """(index of a pair's first value, of its second) of every pair."""
    half = rot // 2
    return [(first + 2 * j, first + 2 * j + 1) if layout == "interleaved" else (first + j, first + half + j)
            for j in range(half)]


def check(q, positions, table, layout, first, weights=None):
    """q [T, H, 128] fp32 array of bf16 values."""
    import dsa_sparse_indexer_gb300 as dsa
    T, H, _ = q.shape
    weights = np.ones((T, H), np.float32) if weights is None else weights
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()   # noqa: E731
    got, got_w = dsa.indexer_query_fp8(cuda(q).bfloat16(), cuda(weights), cuda(np.asarray(positions, np.int32)),
                                       cuda(table), layout=layout, first=first)
    with np.errstate(invalid="ignore", over="ignore"):
        y, _, want_w = IC.queries(q.astype(np.float64), weights.astype(np.float64), 1.0, positions,
                                  table.astype(np.float64), layout, first)
    got, want = got.cpu().numpy(), KF.encode(y)
    assert np.array_equal(got_w.double().cpu().numpy(), want_w)
    assert np.array_equal(got, want), [(tuple(i), y[tuple(i)], got[tuple(i)], want[tuple(i)])
                                       for i in np.argwhere(got != want)[:4]]


@pytest.mark.parametrize("layout,rot,first", TURNS)
def test_infinities_and_the_largest_values_that_turn(layout, rot, first):
    """In the first and the last pair: infinite values, and finite ones that turn
    past fp32's range; beside them ordinary, tiny and infinite carried values."""
    table = RO.table(50, rot, 1e4).astype(np.float32)
    tops = [(INF, 1.0), (1.0, -INF), (-INF, 0.0), (0.0, INF), (INF, INF), (INF, -INF), (3e38, 3e38), (3e38, -3e38),
            (-3e38, 2.5e38), (3.38e38, 3.38e38), (3e38, 1.0), (2e38, INF), (float("nan"), 3e38)]
    turning = {i for pair in pairs_of(layout, rot, first) for i in pair}
    carried = [i for i in range(128) if i not in turning]
    rng = np.random.default_rng(rot + first)
    heads = []
    for a, b in tops:
        for i, j in {pairs_of(layout, rot, first)[0], pairs_of(layout, rot, first)[-1]}:
            for gain in (1.0, 2.0 ** -120, 2.0 ** 120):
                x = rng.standard_normal(128) * gain
                x[i], x[j] = a, b
                heads.append(x)
                if carried:
                    heads.append(x.copy())
                    heads[-1][carried[-1]] = INF
    q = torch.from_numpy(np.array(heads)).bfloat16().float().numpy()
    T = 5
    check(np.tile(q, (T, 1, 1)), [1, 7, 8, 23, 49], table, layout, first)
