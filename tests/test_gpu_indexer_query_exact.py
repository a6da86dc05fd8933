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


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().float().numpy()


def pairs_next_to(targets, table, layout, rng, n, differ):
    """Of n random pairs (position, pair's index, x, partner) whose turned first value
    falls next to one of `targets`, those where fp32 arithmetic, a fused multiply-add
    of a rounded product, differs from the exact value by `differ`."""
    half = table.shape[1] // 2
    pos, j = rng.integers(1, table.shape[0], n), rng.integers(0, half, n)
    c, s = table[pos, j].astype(np.float64), -table[pos, half + j].astype(np.float64)
    p = bf16(rng.choice([-1.0, 1.0], n) * rng.uniform(20, 200, n)).astype(np.float64)
    x = bf16((rng.choice(targets, n) - p * s) / c).astype(np.float64)
    exact, fp32 = x * c + p * s, (x * c + (p * s).astype(np.float32)).astype(np.float32).astype(np.float64)
    hit = differ(exact, fp32) & (np.abs(x) <= 220)
    return [(int(pos[i]), int(j[i]), x[i], p[i]) for i in np.nonzero(hit)[0][:64]]


LAYOUTS = [("half", 64, 0), ("interleaved", 64, 0), ("interleaved", 50, 33), ("half", 64, 64), ("half", 6, 5)]


@pytest.mark.parametrize("T,H", [(None, 3), (1024, 64)])
@pytest.mark.parametrize("layout,rot,first", LAYOUTS)
def test_cancelling_pairs_next_to_a_middle(layout, rot, first, T, H):
    """Small values that two large products leave, next to the middle between two
    codes (the head's scale is 1, set by a carried value)."""
    table = RO.table(300, rot, 1e4).astype(np.float32)
    rng = np.random.default_rng(rot + first)
    grid = KF.decode(np.arange(0x50, dtype=np.uint8))       # 0 to 7.5
    middles = (grid[1:] + grid[:-1]) / 2
    hits = pairs_next_to(np.concatenate([middles, -middles]), table, layout, rng, 1 << 21,
                         lambda exact, fp32: KF.encode(exact) != KF.encode(fp32))
    assert len(hits) >= 16
    T = T or len(hits)
    q = bf16(rng.standard_normal((T, H, 128)))
    turning = {i for pair in pairs_of(layout, rot, first) for i in pair}
    carried = [i for i in range(128) if i not in turning]
    pos = np.zeros(T, np.int64)
    for t in range(T):
        pos[t], j, x, p = hits[t % len(hits)]
        a, b = pairs_of(layout, rot, first)[j]
        q[t, t % H, a], q[t, t % H, b], q[t, t % H, carried[0]] = x, p, 300.0
    check(q, pos, table, layout, first)


@pytest.mark.parametrize("layout,rot,first", LAYOUTS)
def test_largest_values_next_to_a_scale(layout, rot, first):
    """Turned values within fp32's error of 448 times a power of two, the head's
    largest: the scale is the exact value's."""
    table = RO.table(300, rot, 1e4).astype(np.float32)
    rng = np.random.default_rng(rot + first + 1)
    hits = pairs_next_to(np.array([224.0, -224.0]), table, layout, rng, 1 << 21,
                         lambda exact, fp32: (np.abs(exact) <= 224.0) != (np.abs(fp32) <= 224.0))
    assert len(hits) >= 4
    q = np.zeros((len(hits), 2, 128), np.float32)
    for t, (_, j, x, p) in enumerate(hits):
        a, b = pairs_of(layout, rot, first)[j]
        q[t, :, a], q[t, :, b] = x, p
    check(q, [h[0] for h in hits], table, layout, first)


@pytest.mark.parametrize("layout,rot,first", LAYOUTS)
def test_tiny_heads(layout, rot, first):
    """Heads near and below the smallest scale, whose products' errors are subnormal."""
    table = RO.table(300, rot, 1e4).astype(np.float32)
    rng = np.random.default_rng(rot + first + 2)
    q = bf16(rng.standard_normal((64, 66, 128)) * 2.0 ** -np.arange(58, 124)[None, :, None])
    check(q, rng.integers(0, 300, 64), table, layout, first)


def test_a_chunk_of_heads():
    """262144 heads of ordinary values."""
    table = RO.table(4096, 64, 1e4).astype(np.float32)
    rng = np.random.default_rng(11)
    for start in range(0, 4096, 1024):
        q = bf16(rng.standard_normal((1024, 64, 128)))
        w = rng.standard_normal((1024, 64)).astype(np.float32)
        check(q, np.arange(start, start + 1024), table, "half", 0, w)


@pytest.mark.parametrize("layout,rot,first", TURNS)
def test_infinities_at_position_0(layout, rot, first):
    """Position 0 turns by the table's row like any other: beside an infinity a value
    times a sine of 0 is NaN in every layout, and no part of the scale."""
    table = RO.table(3, rot, 1e4).astype(np.float32)
    a, b = pairs_of(layout, rot, first)[-1]
    q = bf16(np.random.default_rng(5).standard_normal((3, 4, 128)))
    q[:, 0, a], q[:, 1, b], q[:, 2, b], q[:, 2, a], q[:, 3, 17] = INF, -INF, INF, 1000.0, INF
    check(q, [0, 1, 0], table, layout, first)
