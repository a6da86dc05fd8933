"""GPU parity of dsa_sparse_mla_decode_fp8 where the blocks of one list have
scales of very different sizes, against the fp64 softmax (oracle/attention.py)
over the cache's values.

Tolerance, from the arithmetic.  A weight times its token's scale, u_j = p_j t_j,
enters the value product as e4m3 plus what that leaves as e5m2, relative to a
reference that brings the largest u to at least 2^3.  (A token of scale 0 has no
product; it counts as one of the least scale, 2^-100, when that is chosen.)
With m the largest u:
 * u >= 2^-6 there: half an e4m3 step leaves 2^-4 u, half an e5m2 step of that
   2^-3: 2^-7 u.  The normaliser takes the weight as it was rounded, so that O
   moves by 2^-7 p_j |v_j - O|.  (m may grow to 2^8.75 before the reference
   moves: such a u is at least 2^-14.75 m.)
 * u < 2^-6 there, so below 2^-9 m: e4m3's steps are 2^-9 and leave at most 2^-10
   and at most u, e5m2 an eighth of that, or half of its least step, 2^-17:
   min(2^-16 m, 2^-3 u) + 2^-20 m.  The normaliser has the weight itself, so O
   moves by that times the codes |c_j|, whatever t_j.
The product is rounded to fp16 before: 2^-11 sum p |v|.  The query's two 8-bit
floats are off by half of e4m3's least step, 2^-10, where the head's largest value
is at least 2^7: 2^-17 of it; sums are fp32 (2^-20 of the sum of magnitudes).  A
score is off by d = |scale| (2^-17 max|q| sum|k| + 2^-20 sum|q k|), which moves
lse2 by d / ln 2 and O by 2 d sum p |v - O|.  1 % covers second orders.  lse2 adds
its own sums (2^-20) and 1e-6 of its size; O is rounded to bf16 (2^-8)."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import attention as OA
from oracle import combine as OC
from oracle import kv_fp8 as KF
from tests import gpu_cases as G

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(192.0)
LEAST = 2.0 ** -100
# (rows, heads): a pair split over a cluster; several pairs a CTA; and with few heads.
FORMS = [(1, 128), (80, 128), (80, 16)]


def _bounds(q, codes, t, out, lse2):
    """(out, lse2) bounds of q [H, 576] over codes [n, 576] times t [n]."""
    rows = codes * t[:, None]
    x = SCALE * (q @ rows.T)
    p = np.exp(x - x.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    u = p * t
    m = (p * np.maximum(t, LEAST)).max(axis=1, keepdims=True)
    v = np.abs(rows[None, :, :512] - out[:, None, :])
    spread = np.einsum("hn,hnd->hd", p, v)
    relative = np.einsum("hn,hnd->hd", np.where(u >= 2.0 ** -15 * m, p, 0), v)
    small = np.where((u > 0) & (u <= 2.0 ** -8.9 * m), np.minimum(2.0 ** -16 * m, 2.0 ** -3 * u) + 2.0 ** -20 * m, 0)
    lost = small @ np.abs(codes[:, :512]) + 2.0 ** -11 * (p @ np.abs(rows[:, :512]))
    d = SCALE * (2.0 ** -17 * np.abs(q).max(axis=1) * np.abs(rows).sum(axis=1).max()
                 + 2.0 ** -20 * (np.abs(q) @ np.abs(rows).T).max(axis=1))
    tol = 2.0 ** -8 * np.abs(out) + 1.01 * (2.0 ** -7 * relative + 2 * d[:, None] * spread + lost)
    return tol, d / np.log(2.0) + 2.0 ** -20 / np.log(2.0) + 1e-6 * np.abs(lse2)


def _compare(rows, H, q, codes, scales, block, order):
    """One list `order` for every row; q [576], the head h's times 1 or as given [H, 576]."""
    import dsa_sparse_indexer_gb300 as dsa
    bits = W.f32_to_bf16_bits(np.broadcast_to(q, (rows, H, 576)).astype(np.float32).copy())
    K = len(order)
    slots = np.tile(order.astype(np.int32), (1, rows, 1))
    counts = torch.full((1, rows), K, dtype=torch.int32, device="cuda")
    err = dsa.new_error_flags("cuda")
    out, lse2 = dsa.sparse_mla_decode_fp8(G.dev(bits.view(np.int16)).view(torch.bfloat16),
                                          G.dev(codes[None]), G.dev(scales[None].astype(np.float32)),
                                          G.dev(slots), counts, SCALE, err_flags=err)
    assert int(err.item()) == 0
    c, t = KF.decode(codes[order]), scales[order // block]
    q64 = OC.bf16_to_f64(bits[0])
    want_o, want_l = OA.sparse_mla_decode(q64, c * t[:, None], SCALE, 512)
    tol_o, tol_l = _bounds(q64, c, t, want_o, want_l)
    for r in sorted({0, rows // 2, rows - 1}):
        got_l = lse2[0, r].double().cpu().numpy()
        assert (np.abs(got_l - want_l) <= tol_l).all(), np.abs(got_l - want_l).max()
        off = np.abs(out[0, r].double().cpu().numpy() - want_o) / (tol_o + 1e-300)
        assert (off <= 1).all(), off.max()


def _codes(rng, n):
    return KF.encode(np.clip(rng.standard_normal((n, 576)) * 60, -448, 448))


@pytest.mark.parametrize("rows,H", FORMS)
@pytest.mark.parametrize("mass,ratio", [(0.9, 64), (0.97, 16), (0.5, 512), (0.5, 1024), (0.999, 2 ** 20)])
def test_many_tokens_of_small_scale_beside_one_of_a_large_one(rows, H, mass, ratio):
    """2000 tokens that share `mass` of the softmax, in blocks whose scale is
    1 / ratio of the remaining token's: their products are small, their share
    of the normaliser is not."""
    rng = np.random.default_rng(ratio)
    n, block, K = 2112, 64, 2001
    codes = _codes(rng, n)
    codes[:, 512:] = 0
    codes[0, 512] = KF.encode(np.array([64.0]))[0]
    scales = np.full(n // block, 1.0 / ratio)
    scales[0] = 1.0
    q = np.zeros(576)
    q[512] = np.log((1 - mass) * 2000.0 / mass) / (SCALE * 64.0)
    order = 64 + rng.permutation(2000)
    order = np.insert(order, 1000, 0)
    assert len(order) == K
    _compare(rows, H, q, codes, scales, block, order)


@pytest.mark.parametrize("rows,H", FORMS)
@pytest.mark.parametrize("size", [2.0 ** -7, 2.0 ** -10, 2.0 ** -40, 2.0 ** -90])
@pytest.mark.parametrize("lead", [0, 10])
def test_blocks_of_scale_zero_beside_others(rows, H, size, lead):
    """Tokens in blocks of scale 0 (score 0, no value) beside tokens of ordinary
    and small scales with scores about as high, or `lead` binades lower: the
    others' weights keep their precision."""
    rng = np.random.default_rng(lead + H)
    n, block = 2048, 64
    codes = _codes(rng, n)
    scales = np.full(n // block, size)
    scales[::3] = 0.0
    codes[:, 512:] = 0
    codes[:, 512] = KF.encode(rng.integers(56, 65, n).astype(np.float64))
    q = np.zeros(576)
    q[512] = -lead * np.log(2.0) / (SCALE * 64.0 * size)
    q[0:512:64] = rng.standard_normal(8) / size / 60
    _compare(rows, H, q, codes, scales, block, rng.permutation(n)[:1000])


@pytest.mark.parametrize("rows,H", FORMS)
def test_a_list_that_begins_or_ends_with_blocks_of_scale_zero(rows, H):
    rng = np.random.default_rng(rows)
    n, block = 1024, 64
    codes, scales = _codes(rng, n), np.full(n // block, 2.0 ** -30)
    scales[:5] = 0.0
    q = rng.standard_normal(576) * 2.0 ** 30 / 60
    first = rng.permutation(320)
    for order in (np.concatenate([first, 320 + rng.permutation(500)]),
                  np.concatenate([320 + rng.permutation(500), first])):
        _compare(rows, H, q, codes, scales, block, order)


@pytest.mark.parametrize("rows,H", FORMS)
@pytest.mark.parametrize("least,most", [(2.0 ** -100, 2.0 ** 100), (2.0 ** -70, 2.0 ** 70), (2.0 ** -100, 2.0 ** 30)])
@pytest.mark.parametrize("rising", [True, False])
def test_the_least_and_the_largest_scale_in_one_list(rows, H, least, most, rising):
    """Tiles (and a split pair's parts) of the least scales, then of the
    largest, with equal scores: every token counts in the normaliser."""
    rng = np.random.default_rng(rows + H)
    n, block = 1024, 64
    codes = _codes(rng, n)
    scales = np.full(n // block, least)
    scales[n // block // 2:] = most
    _compare(rows, H, np.zeros(576), codes, scales, block, np.arange(n) if rising else np.arange(n)[::-1].copy())


@pytest.mark.parametrize("rows,H", FORMS)
def test_query_values_between_the_steps_of_their_second_part(rows, H):
    """Every value halfway between two steps of its 8-bit parts, beside a
    largest one of exactly 2^7: the scores' full bound, all on one side."""
    rng = np.random.default_rng(H)
    n, block = 512, 64
    codes = KF.encode(np.abs(rng.standard_normal((n, 576))) * 60)
    codes[:, 0] = 0
    q = np.full(576, 0.125 * (1 + 1 / 128))
    q[0] = 128.0
    _compare(rows, H, q, codes, np.full(n // block, 2.0 ** -7), block, rng.permutation(n)[:500])
