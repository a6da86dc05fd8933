"""GPU parity of the 8-bit MLA cache: dsa_kv_cache_insert_fp8 bit for bit with
the oracle (oracle/kv_fp8.py), dsa_sparse_mla_decode_fp8 with the fp64 softmax
(oracle/attention.py) over the cache's values, and both in the decode loop.

Attention tolerance, from the arithmetic.  A weight, times its token's scale
t_j, enters the value product as u_j = p_j t_j in two 8-bit floats, the second
holding what the first leaves; the largest u is at least 2^3.
 * u >= 2^-6: e4m3 leaves at most 2^-4 u, of which e5m2 leaves 2^-3: 2^-7 u.
 * u < 2^-6: e4m3's steps are 2^-9 there and it leaves at most 2^-10 and at most
   u, of which e5m2 leaves 2^-3: min(2^-13, 2^-3 u); or half of e5m2's least
   step, 2^-17.
With m the largest u, an error of 2^-13 is at most 2^-16 m, of 2^-17 2^-20 m, so
that p_j is off by at most e_j = 2^-7 p_j + min(2^-16 m / t_j, 2^-3 p_j) +
2^-20 m / t_j.  The normaliser follows these errors: O = sum p v / sum p moves by
at most sum e |v - O| / sum p (first order; 1 % more covers the second).  It does
not follow the rounding of u to fp16 before, half a step 2^-11: 2^-11 sum p |v|.
The query enters the scores as two 8-bit floats with an error below
2^-18 of its head's largest value, and their sums are fp32 (2^-20 of the sum of
magnitudes, over 576 products): a score is off by
d = |scale| (2^-18 max|q| sum|k| + 2^-20 sum|q k|), moving lse2 by d / ln 2 and
O by 2 d sum p |v - O|.  lse2 adds its own fp32 sums (2^-20 relative to the sum
of weights) and rounding (1e-6 of its size); O is rounded to bf16 (2^-8)."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import attention as OA
from oracle import combine as OC
from oracle import kv_fp8 as KF
from oracle import rope as RO
from tests import gpu_cases as G

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(192.0)


def _bf(bits):
    return G.dev(bits.view(np.int16)).view(torch.bfloat16)


# ---- the insert ---------------------------------------------------------------


def _rows(rng, T, spread=4.0):
    x = rng.standard_normal((T, 576)) * 2.0 ** rng.uniform(-spread, spread, (T, 1))
    bits = W.f32_to_bf16_bits(x.astype(np.float32))
    return bits, OC.bf16_to_f64(bits)


def _insert(bits, slots, cache, scales, work=None):
    import dsa_sparse_indexer_gb300 as dsa
    g = G.Guards()
    c = g.empty(cache.shape, torch.uint8)
    s = g.empty(scales.shape, torch.float32)
    c.copy_(G.dev(cache))
    s.copy_(G.dev(scales))
    err = dsa.new_error_flags("cuda")
    dsa.kv_cache_insert_fp8(_bf(np.ascontiguousarray(bits[:, :512])),
                            _bf(np.ascontiguousarray(bits[:, 512:])),
                            G.dev(np.asarray(slots, np.int32)), c, s, work=work, err_flags=err)
    g.check()
    return c.cpu().numpy(), s.cpu().numpy(), int(err.item())


def _same_codes(got, want):
    nan = (want & 0x7F) == 0x7F
    assert np.array_equal((got & 0x7F) == 0x7F, nan)
    assert np.array_equal(got[~nan], want[~nan])


@pytest.mark.parametrize("T", [1, 5, 64, 512, 513, 1500])
@pytest.mark.parametrize("block", [1, 5, 16, 64, 128, 1024])
@pytest.mark.parametrize("state", ["empty", "held"])
def test_insert_matches_the_oracle(T, block, state):
    """Shuffled slots with holes, a slot named twice, blocks that stay; into
    empty blocks, and into held ones whose scales rise for some."""
    rng = np.random.default_rng(T * 7 + block)
    n = 2048 // block * block
    bits, rows = _rows(rng, T)
    slots = rng.permutation(n)[:T] if T <= n else rng.integers(0, n, T)
    slots[::9] = -1
    if T > 12:
        slots[11] = slots[3] = slots[7]
        slots[12], slots[1] = 0, n - 1
    cache = W.e4m3_codes(rng, (n, 576))
    scales = np.zeros(n // block, np.float32)
    if state == "held":
        scales[:] = 2.0 ** rng.integers(-9, -3, n // block)
        scales[rng.random(n // block) < 0.2] = 0.0
    want_c, want_s = KF.insert(cache, scales, rows, slots)
    got_c, got_s, err = _insert(bits, slots, cache, scales)
    assert err == 0
    np.testing.assert_array_equal(got_s, want_s)
    _same_codes(got_c, want_c)


@pytest.mark.parametrize("T,n,block", [
    (700, 4096, 16), (2433, 16384, 64), (3000, 16384, 16), (6000, 32768, 64), (2600, 20800, 1),
    (6000, 16384, 16), (5000, 16384, 32), (4096, 16384, 27), (4095, 16384, 64), (2048, 2048, 1024),
    (4000, 24576, 256)])
@pytest.mark.parametrize("order", ["prompt", "any"])
def test_insert_of_many_rows(T, n, block, order):
    """Both ways of finding the blocks of a large call, on both sides of the
    sizes that choose; tokens in the order of their slots, or in none."""
    rng = np.random.default_rng(T + block)
    n = n // block * block
    bits, rows = _rows(rng, T)
    if order == "prompt":
        blocks = rng.permutation(n // block)
        slots = (blocks[:, None] * block + np.arange(block)).reshape(-1)[:T].copy()
    else:
        slots = rng.integers(0, n, T)
    slots[::13] = -1
    slots[5] = slots[T - 2]
    cache = W.e4m3_codes(rng, (n, 576))
    scales = 2.0 ** rng.integers(-9, -3, n // block).astype(np.float32)
    scales[rng.random(n // block) < 0.2] = 0.0
    want_c, want_s = KF.insert(cache, scales, rows, slots)
    got_c, got_s, err = _insert(bits, slots, cache, scales)
    assert err == 0
    np.testing.assert_array_equal(got_s, want_s)
    _same_codes(got_c, want_c)


@pytest.mark.parametrize("T", [40, 600])
def test_insert_of_extreme_values(T):
    """Infinities, NaN, zero rows, the smallest and largest bf16, scales that
    are no power of two, negative or NaN scales (empty blocks), slots past the
    cache."""
    rng = np.random.default_rng(T)
    n, block = 1024, 16
    bits, _ = _rows(rng, T, spread=1.0)
    bits[0] = 0
    bits[1, 5], bits[1, 6], bits[1, 570] = 0x7F80, 0xFF80, 0x7FC1
    bits[2] = 0x0001
    bits[3, 3] = 0x7F7F
    bits[4] = 0x8000
    bits[5] = 0x7F80
    slots = rng.permutation(n)[:T]
    slots[6], slots[7] = n, 2 ** 31 - 1
    cache = W.e4m3_codes(rng, (n, 576))
    cache[:, 0] = 0x7F
    scales = rng.uniform(0.001, 0.01, n // block).astype(np.float32)
    scales[3], scales[4], scales[5] = -1.0, np.nan, 0.0
    want_c, want_s = KF.insert(cache, scales, OC.bf16_to_f64(bits), slots)
    got_c, got_s, err = _insert(bits, slots, cache, scales)
    assert err == 1
    np.testing.assert_array_equal(got_s, want_s)
    _same_codes(got_c, want_c)


def test_insert_with_any_contents_in_the_workspace():
    """The words a large call leaves, or any others, do not disturb the next."""
    rng = np.random.default_rng(11)
    n, block, T = 4096, 64, 700
    cache, scales = W.e4m3_codes(rng, (n, 576)), np.full(n // block, 2.0 ** -7, np.float32)
    work = torch.randint(-5, 720, (n + n // block,), dtype=torch.int32, device="cuda")
    for k in range(3):
        bits, rows = _rows(rng, T)
        slots = rng.permutation(n)[:T]
        want_c, want_s = KF.insert(cache, scales, rows, slots)
        cache, scales, err = _insert(bits, slots, cache, scales, work=work)
        assert err == 0
        np.testing.assert_array_equal(scales, want_s)
        _same_codes(cache, want_c)


def test_insert_one_token_at_a_time_into_a_page_captured():
    """A page filled by decode steps of one replayed graph."""
    import dsa_sparse_indexer_gb300 as dsa
    rng = np.random.default_rng(12)
    bits, rows = _rows(rng, 64)
    kv, kpe = torch.empty((1, 512), dtype=torch.bfloat16, device="cuda"), \
        torch.empty((1, 64), dtype=torch.bfloat16, device="cuda")
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = torch.zeros((128, 576), dtype=torch.uint8, device="cuda")
    scales = torch.zeros(2, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.kv_cache_insert_fp8(kv, kpe, slot, cache, scales)
    want_c, want_s = np.zeros((128, 576), np.uint8), np.zeros(2, np.float32)
    order = rng.permutation(64) + 64
    for t in range(64):
        kv.copy_(_bf(bits[t:t + 1, :512]))
        kpe.copy_(_bf(bits[t:t + 1, 512:]))
        slot.fill_(int(order[t]))
        graph.replay()
        want_c, want_s = KF.insert(want_c, want_s, rows[t:t + 1], order[t:t + 1])
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
    _same_codes(cache.cpu().numpy(), want_c)


def test_insert_refusals():
    import dsa_sparse_indexer_gb300 as dsa
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")      # noqa: E731
    i32, u8, f32 = torch.int32, torch.uint8, torch.float32
    with pytest.raises(ValueError, match="whole number"):
        dsa.kv_cache_insert_fp8(z(1, 512), z(1, 64), z(1, t=i32), z(100, 576, t=u8), z(3, t=f32))
    with pytest.raises(ValueError, match="T slots"):
        dsa.kv_cache_insert_fp8(z(2, 512), z(1, 64), z(1, t=i32), z(64, 576, t=u8), z(1, t=f32))
    with pytest.raises(ValueError, match="work"):
        dsa.kv_cache_insert_fp8(z(1, 512), z(1, 64), z(1, t=i32), z(64, 576, t=u8), z(1, t=f32),
                                work=z(64, t=i32))
    with pytest.raises(TypeError, match="uint8"):
        dsa.kv_cache_insert_fp8(z(1, 512), z(1, 64), z(1, t=i32), z(64, 576), z(1, t=f32))
    with pytest.raises(dsa.DSAError):
        dsa.kv_cache_insert_fp8(z(1, 512), z(1, 64), z(1, t=i32), z(2048, 576, t=u8), z(1, t=f32))


# ---- the attention --------------------------------------------------------------


def _tolerance(q, rows, scale, out, lse2, t=None):
    """(out, lse2) bounds of one (shard, row): q [H, 576], rows [n, 576], t [n] the
    rows' scales (all alike when not given)."""
    x = scale * (q @ rows.T)
    p = np.exp(x - x.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    v = np.abs(rows[None, :, :512] - out[:, None, :])                  # [H, n, 512]
    spread = np.einsum("hn,hnd->hd", p, v)
    t = np.ones(len(rows)) if t is None else t.astype(np.float64)
    m = (p * t).max(axis=1, keepdims=True) / t                         # m / t_j
    lost = np.einsum("hn,hnd->hd", np.minimum(2.0 ** -16 * m, 2.0 ** -3 * p) + 2.0 ** -20 * m, v)
    lost += 2.0 ** -11 * (p @ np.abs(rows[:, :512]))
    d = abs(scale) * (2.0 ** -18 * np.abs(q).max(axis=1) * np.abs(rows).sum(axis=1).max()
                      + 2.0 ** -20 * (np.abs(q) @ np.abs(rows).T).max(axis=1))
    tol = 2.0 ** -8 * np.abs(out) + 1.01 * ((2.0 ** -7 + 2 * d[:, None]) * spread + lost) + 1e-30
    return tol, d / np.log(2.0) + 2.0 ** -20 / np.log(2.0) + 1e-6 * np.abs(lse2)


def _attend(q_bits, codes, scales, slots, counts, scale=SCALE):
    import dsa_sparse_indexer_gb300 as dsa
    err = dsa.new_error_flags("cuda")
    g = G.Guards()
    S, rows = counts.shape
    H = q_bits.shape[1]
    out, lse2 = dsa.sparse_mla_decode_fp8(_bf(q_bits), G.dev(codes), G.dev(scales),
                                          G.dev(slots.astype(np.int32)),
                                          G.dev(counts.astype(np.int32)), scale,
                                          out=g.empty((S, rows, H, 512), torch.bfloat16),
                                          lse2=g.empty((S, rows, H), torch.float32), err_flags=err)
    g.check()
    return (OC.bf16_to_f64(out.view(torch.int16).cpu().numpy().view(np.uint16)),
            lse2.cpu().numpy().astype(np.float64), int(err.item()))


def _check(q_bits, values, slots, counts, scale, out, lse2, pairs=None, scales=None):
    """values: [S, n_slots, 576] fp64, or a function of (shard, slots); scales:
    [S, blocks], where they are not all alike."""
    q = OC.bf16_to_f64(q_bits)
    S, R = counts.shape
    at = values if callable(values) else (lambda s, j: values[s, j])
    for s, r in (pairs if pairs is not None else np.ndindex(S, R)):
        sel = slots[s, r, :counts[s, r]]
        if len(sel) == 0:
            assert (out[s, r] == 0).all() and np.isneginf(lse2[s, r]).all(), (s, r)
            continue
        rows = at(s, sel)
        want_o, want_l = OA.sparse_mla_decode(q[r], rows, scale, 512)
        t = None if scales is None else scales[s, sel // (values.shape[1] // scales.shape[1])]
        tol_o, tol_l = _tolerance(q[r], rows, scale, want_o, want_l, t)
        off = np.abs(out[s, r] - want_o) / tol_o
        assert (off <= 1).all(), (s, r, off.max(), np.argwhere(off > 1)[:4])
        assert (np.abs(lse2[s, r] - want_l) <= tol_l).all(), (s, r, np.abs(lse2[s, r] - want_l).max())


def _cache(rng, S, n_slots, block, pow2):
    codes = KF.encode(np.clip(rng.standard_normal((S, n_slots, 576)) * 60, -448, 448))
    scales = np.exp2(rng.normal(0, 0.7, (S, n_slots // block))) / 60
    if pow2:
        scales = 2.0 ** np.round(np.log2(scales))
    return codes, scales.astype(np.float32)


@pytest.mark.parametrize("H,block", [(1, 64), (8, 1), (16, 16), (40, 48), (64, 64), (96, 100),
                                     (128, 64), (192, 128), (130, 64)])
def test_random_slot_sets(H, block):
    """Counts around every tile boundary, from none to a long list."""
    rng = np.random.default_rng(H)
    S, R, K = 3, 5, 1100
    n_slots = 2400 // block * block
    codes, scales = _cache(rng, S, n_slots, block, pow2=H % 32 == 0)
    q = W.mla_query(R, H, seed=10 + H)
    counts = np.array([[0, 1, 31, 32, 33], [127, 128, 129, 255, 1100], [257, 64, 0, 640, 2]])
    slots = np.full((S, R, K), -1, np.int64)
    for s, r in np.ndindex(S, R):
        slots[s, r, :counts[s, r]] = rng.choice(n_slots, counts[s, r], replace=False)
    out, lse2, err = _attend(q, codes, scales, slots, counts)
    assert err == 0
    _check(q, KF.values(codes, scales), slots, counts, SCALE, out, lse2, scales=scales)


@pytest.mark.parametrize("rows,S,K", [(1, 1, 1), (1, 1, 2048), (2, 1, 2048), (1, 3, 777),
                                      (37, 1, 300), (160, 2, 200)])
def test_few_and_many_rows(rows, S, K):
    """Whatever way the work is split over the GPU: a single row to more rows
    than it holds at once."""
    rng = np.random.default_rng(rows + K)
    H, n_slots = 128, 4096
    codes, scales = _cache(rng, S, n_slots, 64, True)
    q = W.mla_query(rows, H, seed=rows)
    counts = rng.integers(K // 2, K + 1, (S, rows))
    counts[0, 0] = K
    slots = rng.integers(0, n_slots, (S, rows, K))       # slots repeat: each counts
    out, lse2, err = _attend(q, codes, scales, slots, counts)
    assert err == 0
    pairs = None if rows * S <= 8 else [(s, r) for s in range(S) for r in rng.integers(0, rows, 4)]
    _check(q, KF.values(codes, scales), slots, counts, SCALE, out, lse2, pairs, scales)


@pytest.mark.parametrize("H", [1, 16, 17, 32, 33, 48])
def test_few_heads_many_rows(H):
    """Many pairs a CTA, with idle softmax warps: lists from none to four tiles,
    rows with nothing on any shard, one pair between new rows."""
    rng = np.random.default_rng(H)
    rows, S, K, n_slots = 250, 3, 400, 4096
    codes, scales = _cache(rng, S, n_slots, 64, False)
    q = W.mla_query(rows, H, seed=H)
    counts = rng.integers(1, K + 1, (S, rows))
    counts[:, ::3] = rng.integers(0, 130, counts[:, ::3].shape)
    counts[rng.random((S, rows)) < 0.2] = 0
    counts[:, 7:9] = 0
    counts[1:, 40:60] = 0
    slots = rng.integers(0, n_slots, (S, rows, K))
    out, lse2, err = _attend(q, codes, scales, slots, counts)
    assert err == 0
    pairs = [(s, r) for s in range(S) for r in list(range(0, 12)) + list(range(40, 250, 9))]
    _check(q, KF.values(codes, scales), slots, counts, SCALE, out, lse2, pairs, scales)
    again, lse2_again, _ = _attend(q, codes, scales, slots, counts)
    assert np.array_equal(out, again) and np.array_equal(lse2, lse2_again)


@pytest.mark.parametrize("rows,K", [(1, 2048), (3, 700)])
def test_few_rows_without_a_workspace(rows, K):
    """The C entry point with work = NULL does not split the lists; with it,
    the parts' sum is within the same bounds, and any contents do."""
    from dsa_sparse_indexer_gb300 import _lib
    rng = np.random.default_rng(rows)
    S, H, n_slots = 1, 100, 4096
    codes, scales = _cache(rng, S, n_slots, 64, True)
    q = W.mla_query(rows, H, seed=rows)
    counts = np.full((S, rows), K)
    counts[0, -1] = K // 2 + 5
    slots = rng.integers(0, n_slots, (S, rows, K))
    need = _lib.load().dsa_sparse_mla_decode_fp8_work(rows, S, H, K)
    assert need > 0
    args = [_bf(q), G.dev(codes), G.dev(scales), G.dev(slots.astype(np.int32)),
            G.dev(counts.astype(np.int32))]
    for work in (None, torch.full((need // 4,), float("nan"), device="cuda")):
        g = G.Guards()
        out, lse2 = g.empty((S, rows, H, 512), torch.bfloat16), g.empty((S, rows, H), torch.float32)
        P = lambda t: None if t is None else t.data_ptr()      # noqa: E731
        _lib.call("dsa_sparse_mla_decode_fp8", P(args[0]), P(args[1]), P(args[2]), n_slots, 64,
                  P(args[3]), P(args[4]), rows, S, H, K, SCALE, P(out), P(lse2), P(work), None,
                  torch.cuda.current_stream().cuda_stream)
        g.check()
        _check(q, KF.values(codes, scales), slots, counts, SCALE,
               OC.bf16_to_f64(out.view(torch.int16).cpu().numpy().view(np.uint16)),
               lse2.double().cpu().numpy())


def _left_out_case():
    rng = np.random.default_rng(9)
    S, R, H, K, n_slots = 2, 3, 64, 512, 640
    codes, scales = _cache(rng, S, n_slots, 64, True)
    slots = rng.integers(64, 576, (S, R, K))
    counts = np.array([[40, 200, K], [3, 130, 5]])
    bad = [(0, 0, 5, n_slots), (0, 0, 39, -1), (0, 1, 150, -7), (1, 0, 0, 2 ** 31 - 1),
           (1, 1, 129, n_slots + 1)]
    bad += [(1, 2, j, -1) for j in range(5)]             # a row with nothing left
    bad += [(0, 2, j, -1) for j in range(128, 256)]      # a whole tile left out
    return rng, S, R, H, K, n_slots, codes, scales, slots, counts, bad


def test_slots_left_out_do_not_reach_the_result():
    """Bad slots below the count are flagged and left out; the cache around
    the selected rows (its first and last blocks among it) holds NaN codes, and
    the blocks' scales there NaN and infinity."""
    rng, S, R, H, K, n_slots, codes, scales, slots, counts, bad = _left_out_case()
    for s, r, j, v in bad:
        slots[s, r, j] = v
    codes[:, :64] = codes[:, 576:] = 0x7F
    scales[:, 0], scales[:, 9] = np.nan, np.inf
    used = np.zeros((S, n_slots), bool)
    keep, cnt = np.full_like(slots, -1), np.zeros_like(counts)
    for s, r in np.ndindex(S, R):
        row = slots[s, r, :counts[s, r]]
        row = row[(row >= 0) & (row < n_slots)]
        used[s, row] = True
        cnt[s, r], keep[s, r, :len(row)] = len(row), row
    codes[~used] = 0xFF
    q = W.mla_query(R, H, seed=1)
    out, lse2, err = _attend(q, codes, scales, slots, counts)
    assert err == 1
    values = KF.decode(codes) * np.repeat(np.where(np.isfinite(scales), scales, 0), 64, 1)[..., None]
    _check(q, values, keep, cnt, SCALE, out, lse2)


def test_what_is_not_finite_stays_in_its_head_and_row():
    """An infinity or NaN in a head of the query makes that head's outputs NaN,
    a NaN code in a selected row that row's, and no others."""
    rng = np.random.default_rng(19)
    codes, scales = _cache(rng, 1, 512, 64, True)
    q = W.mla_query(3, 70, seed=6)
    q[0, 2, 7], q[0, 69, 575], q[1, 0, 0] = 0x7F80, 0xFF80, 0x7FC0
    slots = rng.integers(0, 256, (1, 3, 200))
    slots[0, 2, 150] = 300
    codes[0, 300, 40] = 0x7F
    counts = np.array([[200, 130, 200]])
    out, lse2, err = _attend(q, codes, scales, slots, counts)
    assert err == 0
    hit = np.zeros((3, 70), bool)
    hit[0, [2, 69]] = hit[1, 0] = hit[2] = True
    assert np.array_equal(np.isnan(lse2[0]), hit)
    assert np.array_equal(np.isnan(out[0]).any(-1), hit)
    assert np.isnan(out[0][0, [2, 69]]).all() and np.isnan(out[0][1, 0]).all()
    held = q.copy()
    held[0, [2, 69]] = held[1, 0] = 0
    want = [OA.sparse_mla_decode(OC.bf16_to_f64(held[r]), KF.values(codes, scales)[0, slots[0, r, :n]],
                                 SCALE, 512) for r, n in ((0, 200), (1, 130))]
    for r, (o, l) in enumerate(want):
        rows = KF.values(codes, scales)[0, slots[0, r, :counts[0, r]]]
        tol_o, tol_l = _tolerance(OC.bf16_to_f64(held[r]), rows, SCALE, o, l)
        keep = ~hit[r]
        assert (np.abs(out[0, r] - o) <= tol_o)[keep].all()
        assert (np.abs(lse2[0, r] - l) <= tol_l)[keep].all()


@pytest.mark.parametrize("value", [2.0 ** -100, 2.0 ** 100, 2.0 ** -101, 2.0 ** 101, -1.0])
def test_block_scales_at_the_edges(value):
    """Scales from 2^-100 to 2^100 are exact; others in a selected row's block
    are flagged, 0 (an empty block's) is not."""
    rng = np.random.default_rng(20)
    codes, scales = _cache(rng, 1, 256, 64, True)
    q = (rng.standard_normal((1, 16, 576)) / value if value > 0 else rng.standard_normal((1, 16, 576)))
    bits = W.f32_to_bf16_bits(q.astype(np.float32) / 60)
    slots = rng.integers(0, 256, (1, 1, 180))
    out, lse2, err = _attend(bits, codes, np.full((1, 4), value, np.float32), slots, np.array([[180]]))
    inside = 2.0 ** -100 <= value <= 2.0 ** 100
    assert err == (0 if inside else 1)
    if inside:
        _check(bits, KF.values(codes, np.full((1, 4), value)), slots, np.array([[180]]), SCALE, out, lse2)
    out, lse2, err = _attend(bits, codes, np.zeros((1, 4), np.float32), slots, np.array([[180]]))
    assert err == 0 and (out == 0).all()
    np.testing.assert_allclose(lse2, np.log2(180.0), rtol=1e-6)


def test_counts_outside_the_list_are_clamped_and_flagged():
    rng = np.random.default_rng(10)
    codes, scales = _cache(rng, 1, 256, 64, True)
    q = W.mla_query(2, 16, seed=2)
    slots = rng.integers(0, 256, (1, 2, 40))
    out, lse2, err = _attend(q, codes, scales, slots, np.array([[41, -3]]))
    assert err == 1
    _check(q, KF.values(codes, scales), slots, np.array([[40, 0]]), SCALE, out, lse2)


@pytest.mark.parametrize("scale", [-SCALE, 0.0, 1.0, 1e-6])
def test_other_softmax_scales(scale):
    """Negative, zero (every weight 1: the plain mean), steep and flat."""
    rng = np.random.default_rng(13)
    S, R, H, K, n_slots = 2, 2, 128, 400, 1024
    codes, scales = _cache(rng, S, n_slots, 64, False)
    q = W.mla_query(R, H, seed=3)
    counts = np.array([[400, 300], [129, 1]])
    slots = rng.integers(0, n_slots, (S, R, K))
    out, lse2, err = _attend(q, codes, scales, slots, counts, scale=scale)
    assert err == 0
    _check(q, KF.values(codes, scales), slots, counts, scale, out, lse2)
    if scale == 0.0:
        np.testing.assert_allclose(lse2, np.log2(counts)[:, :, None] * np.ones(H), rtol=1e-6)


@pytest.mark.parametrize("rising", [True, False])
def test_maxima_that_keep_moving(rising):
    """Scores that rise by hundreds from tile to tile (the running reference
    moves each time, everything before vanishes), or fall; heads of very
    different sizes, among them a zero query and one of tiny values."""
    rng = np.random.default_rng(14)
    S, R, H, K, n_slots = 1, 1, 64, 1024, 1024
    codes, scales = _cache(rng, S, n_slots, 64, True)
    q = rng.standard_normal((R, H, 576)) * 2.0 ** rng.integers(-12, 4, (R, H, 1))
    q[0, 3] = 0.0
    q[0, 4] *= 1e-30
    q[0, 5, 100] = 300.0
    order = np.argsort(rng.uniform(0, 1, n_slots))[:K]
    main = KF.values(codes, scales)[0, order] @ q[0, 0]
    order = order[np.argsort(main if rising else -main)]
    bits = W.f32_to_bf16_bits(q.astype(np.float32))
    counts = np.array([[K]])
    out, lse2, err = _attend(bits, codes, scales, order[None, None], counts, scale=3.0)
    assert err == 0
    _check(bits, KF.values(codes, scales), order[None, None], counts, 3.0, out, lse2)


def test_many_small_weights_beside_a_large_one():
    """One token with half the weight and two thousand that share the rest:
    none of the small ones may vanish."""
    rng = np.random.default_rng(15)
    K, H = 2001, 16
    codes, scales = _cache(rng, 1, 2048, 64, True)
    codes[0, :, 512:] = KF.encode(np.zeros(64))
    codes[0, 0, 512] = KF.encode(np.array([64.0]))[0]
    scales[:] = 1.0 / 64
    codes[0, :, 1:512] = KF.encode(rng.uniform(0.5, 1.0, (2048, 511)) * 64)
    q = np.zeros((1, H, 576))
    q[0, :, 512] = np.log(2000.0) / SCALE
    bits = W.f32_to_bf16_bits(q.astype(np.float32))
    slots = np.arange(K)[None, None]
    out, lse2, err = _attend(bits, codes, scales, slots, np.array([[K]]))
    assert err == 0
    _check(bits, KF.values(codes, scales), slots, np.array([[K]]), SCALE, out, lse2)


def test_a_cache_longer_than_32_bit_offsets():
    """9 million slots (5.2 GB): rows at its far end."""
    rng = np.random.default_rng(16)
    n_slots, block, K, H = 9_000_000, 1000, 300, 64
    codes = torch.zeros((1, n_slots, 576), dtype=torch.uint8, device="cuda")
    scales = torch.full((1, n_slots // block), 1 / 64, device="cuda")
    sel = np.concatenate([n_slots - 1 - rng.permutation(1000)[:K - 2], [0, n_slots // 2]])
    held = KF.encode(np.clip(rng.standard_normal((K, 576)) * 60, -448, 448))
    codes[0, torch.from_numpy(sel).cuda()] = G.dev(held)
    import dsa_sparse_indexer_gb300 as dsa
    q = W.mla_query(1, H, seed=4)
    out, lse2 = dsa.sparse_mla_decode_fp8(_bf(q), codes, scales, G.dev(sel.astype(np.int32)[None, None]),
                                          G.dev(np.array([[K]], np.int32)), SCALE)
    lookup = {int(s): i for i, s in enumerate(sel)}
    values = lambda s, j: KF.decode(held[[lookup[int(i)] for i in j]]) / 64     # noqa: E731
    _check(q, values, sel[None, None], np.array([[K]]), SCALE,
           OC.bf16_to_f64(out.view(torch.int16).cpu().numpy().view(np.uint16)),
           lse2.double().cpu().numpy())
    # and an insert there
    bits, rows = _rows(rng, 3)
    where = np.array([n_slots - 1, n_slots - 2, 5], np.int32)
    dsa.kv_cache_insert_fp8(_bf(np.ascontiguousarray(bits[:, :512])),
                            _bf(np.ascontiguousarray(bits[:, 512:])), G.dev(where), codes[0], scales[0])
    want_s = [max(1 / 64, KF.scale_for(np.abs(rows[:2]).max())), max(1 / 64, KF.scale_for(np.abs(rows[2]).max()))]
    got = codes[0, torch.from_numpy(where.astype(np.int64)).cuda()].cpu().numpy()
    _same_codes(got[:2], KF.encode(rows[:2] / want_s[0]))
    _same_codes(got[2], KF.encode(rows[2] / want_s[1]))


def test_the_same_call_twice_on_two_streams_and_captured():
    """Two calls at once on two streams, and a captured one replayed with other
    inputs: the same bits as alone."""
    import dsa_sparse_indexer_gb300 as dsa
    rng = np.random.default_rng(17)
    S, R, H, K, n_slots = 2, 40, 128, 512, 4096
    codes, scales = _cache(rng, S, n_slots, 64, True)
    dc, ds = G.dev(codes), G.dev(scales)
    calls = []
    for k in range(2):
        counts = rng.integers(0, K + 1, (S, R)).astype(np.int32)
        slots = rng.integers(0, n_slots, (S, R, K)).astype(np.int32)
        calls.append((_bf(W.mla_query(R, H, seed=20 + k)), G.dev(slots), G.dev(counts)))
    alone = [dsa.sparse_mla_decode_fp8(q, dc, ds, sl, ct, SCALE) for q, sl, ct in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for st, (q, sl, ct) in zip(streams, calls):
        with torch.cuda.stream(st):
            got.append(dsa.sparse_mla_decode_fp8(q, dc, ds, sl, ct, SCALE))
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    q, sl, ct = (t.clone() for t in calls[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse2 = dsa.sparse_mla_decode_fp8(q, dc, ds, sl, ct, SCALE)
    for k in (1, 0):
        for t, new in zip((q, sl, ct), calls[k]):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, alone[k][0]) and torch.equal(lse2, alone[k][1])


def test_attention_refusals():
    import dsa_sparse_indexer_gb300 as dsa
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")      # noqa: E731
    i32, u8, f32 = torch.int32, torch.uint8, torch.float32
    good = dict(q=z(2, 16, 576), kv_cache=z(1, 64, 576, t=u8), block_scales=z(1, 1, t=f32),
                slots=z(1, 2, 8, t=i32), counts=z(1, 2, t=i32), scale=0.1)
    dsa.sparse_mla_decode_fp8(**good)
    for bad, kind in [(dict(q=z(2, 16, 512)), ValueError), (dict(kv_cache=z(1, 64, 576)), TypeError),
                      (dict(block_scales=z(1, 3, t=f32)), ValueError),
                      (dict(block_scales=z(2, 1, t=f32)), ValueError),
                      (dict(slots=z(1, 3, 8, t=i32)), ValueError),
                      (dict(counts=z(2, 1, t=i32)), ValueError),
                      (dict(out=z(1, 2, 16, 576)), ValueError),
                      (dict(lse2=z(1, 2, 17, t=f32)), ValueError),
                      (dict(q=z(2, 576, 16).transpose(1, 2)), ValueError),
                      (dict(scale=float("inf")), dsa.DSAError)]:
        with pytest.raises(kind):
            dsa.sparse_mla_decode_fp8(**{**good, **bad})
    assert dsa.sparse_mla_decode_fp8(**{**good, "q": z(0, 16, 576), "slots": z(1, 0, 8, t=i32),
                                        "counts": z(1, 0, t=i32)})[0].shape == (1, 0, 16, 512)


# ---- together -------------------------------------------------------------------


def test_the_decode_loop_on_an_8_bit_cache():
    """As they are used: a scaled table, prompt keys normed and rotated
    (fused_norm_rope) and inserted in 8 bits on every shard, the queries' tails
    rotated into place, attention over each shard's selected slots, and the
    shards' outputs combined, against the oracles of every step."""
    import dsa_sparse_indexer_gb300 as dsa
    from oracle import pcp_prefill as PP
    S, T, rows, H, block, n_slots = 2, 900, 4, 64, 64, 1024
    rng = np.random.default_rng(21)
    table = dsa.rope_table(4096, 64, scaling="yarn", factor=8.0, orig_max_pos=512)
    cs = table.cpu().numpy()
    assert np.abs(cs - RO.table(4096, 64, 1e4, scaling="yarn", factor=8.0, orig_max_pos=512)).max() < 4e-7
    kv, kpe, w = W.pcp_token_inputs(T, seed=22)
    pos = rng.permutation(4096)[:T].astype(np.int32)
    err = dsa.new_error_flags("cuda")
    kv_rows, kpe_rows = dsa.fused_norm_rope(_bf(kv), _bf(kpe), G.dev(pos), G.dev(w), 1e-6, table,
                                            err_flags=err)
    cache = torch.zeros((S, n_slots, 576), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((S, n_slots // block), device="cuda")
    want_c, want_s = np.zeros((S, n_slots, 576), np.uint8), np.zeros((S, n_slots // block), np.float32)
    rows_f = np.concatenate([OC.bf16_to_f64(t.view(torch.int16).cpu().numpy().view(np.uint16))
                             for t in (kv_rows, kpe_rows)], axis=1)
    ref_kv, ref_kpe = PP.fused_norm_rope(OC.bf16_to_f64(kv), OC.bf16_to_f64(kpe), w, 1e-6, pos, cs)
    assert np.abs(rows_f - np.concatenate([ref_kv, ref_kpe], 1)).max() < 0.05
    for s in range(S):
        mapping = np.full(T, -1, np.int32)
        mapping[s::S] = rng.permutation(n_slots)[:len(mapping[s::S])]
        for a, b in ((0, 600), (600, 601), (601, T)):        # a prompt, a token, the rest
            dsa.kv_cache_insert_fp8(kv_rows[a:b], kpe_rows[a:b], G.dev(mapping[a:b]), cache[s],
                                    scales[s], err_flags=err)
            want_c[s], want_s[s] = KF.insert(want_c[s], want_s[s], rows_f[a:b], mapping[a:b])
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
    _same_codes(cache.cpu().numpy(), want_c)
    # the query: latent part as given, rope part rotated from the projection's tail
    proj = _bf(W.mla_query(rows, H, seed=23))[..., :192].contiguous()
    q = _bf(W.mla_query(rows, H, seed=24)).clone()
    qpos = rng.integers(0, 4096, rows).astype(np.int32)
    dsa.rotary_embed(proj[..., 128:], G.dev(qpos), table, out=q[..., 512:], err_flags=err)
    q_bits = q.view(torch.int16).cpu().numpy().view(np.uint16)
    rotated = RO.rotate(proj[..., 128:].double().cpu().numpy(), qpos, cs, "interleaved")
    assert (np.abs(OC.bf16_to_f64(q_bits[..., 512:]) - rotated) <= 2.0 ** -8 * np.abs(rotated) + 1e-5).all()
    counts = np.array([[300, 0, 1, 128], [256, 0, 129, 450]])
    slots = rng.integers(0, n_slots, (S, rows, 512))
    out, lse2 = dsa.sparse_mla_decode_fp8(q, cache, scales, G.dev(slots.astype(np.int32)),
                                          G.dev(counts.astype(np.int32)), SCALE, err_flags=err)
    ob = OC.bf16_to_f64(out.view(torch.int16).cpu().numpy().view(np.uint16))
    _check(q_bits, KF.values(want_c, want_s), slots, counts, SCALE, ob, lse2.double().cpu().numpy())
    y, lse = dsa.lse_combine(out, lse2, err_flags=err)
    want_y, _ = OC.lse_combine(ob, lse2.cpu().numpy())
    got_y = OC.bf16_to_f64(y.view(torch.int16).cpu().numpy().view(np.uint16))
    assert (np.abs(got_y - want_y) <= G.combine_tolerance(want_y)).all()
    assert int(err.item()) == 0 and torch.isneginf(lse[1]).all()
