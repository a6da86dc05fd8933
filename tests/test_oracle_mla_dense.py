"""The whole-context attention oracle against its own identities."""
import numpy as np
import pytest

from oracle import combine as OC
from oracle import indexer_cache as IC
from oracle import kv_fp8 as KF
from oracle import mla_dense as MD
from oracle import rope as RO


def test_shards_combine_to_the_whole():
    """The shards' parts, merged by their lse2, are attention over the request's
    tokens in order; a tree mask of prefixes is the chain."""
    rng = np.random.default_rng(1)
    S, I, H, b = 4, 2, 2, 16
    lens, starts = [37, 5], [0, 3, 4]
    table = np.stack([rng.permutation(4).reshape(2, 2) for _ in range(S)]).astype(np.int32)
    cache = rng.standard_normal((S, 4 * b, 576))
    q = rng.standard_normal((4, H, 576))
    out, lse2, *_ = MD.decode(q, cache, table, b, starts, lens, S, I, 0.07)
    whole, lse = OC.lse_combine(out, lse2.astype(np.float32))
    for r, row, last in ((0, 0, 34), (0, 2, 36), (1, 3, 4)):
        t = np.arange(last + 1)
        loc = t // (I * S) * I + t % I
        k = cache[(t // I) % S, table[(t // I) % S, r, loc // b] * b + loc % b]
        x = q[row] @ k.T * 0.07
        w = np.exp(x - x.max(1, keepdims=True))
        assert np.allclose(whole[row], w @ k[:, :512] / w.sum(1, keepdims=True), atol=1e-6)
    mask = np.array([[1], [3], [7], [1]], np.int32)
    again, again2, *_ = MD.decode(q, cache, table, b, starts, lens, S, I, 0.07, tree_mask=mask)
    assert np.array_equal(again, out) and np.array_equal(again2, lse2)


def test_tree_bits_past_the_words_and_empty_rows():
    rng = np.random.default_rng(2)
    cache = rng.standard_normal((1, 64, 576))
    table = np.arange(4, dtype=np.int32).reshape(1, 1, 4)
    q = rng.standard_normal((40, 1, 576))
    mask = np.zeros((40, 1), np.int32)
    mask[39, 0] = -1 << 31                       # token 31 alone
    out, lse2, *_ = MD.decode(q, cache, table, 16, [0, 40], [40], 1, 1, 0.1, tree_mask=mask)
    assert np.isneginf(lse2[0, :39]).all() and (out[0, :39] == 0).all()
    assert np.allclose(out[0, 39, 0], cache[0, 31, :512])


def test_prefill_is_decode_of_a_chain():
    rng = np.random.default_rng(3)
    q, kn, v = rng.standard_normal((3, 2, 192)), rng.standard_normal((5, 2, 128)), rng.standard_normal((5, 2, 128))
    pe = rng.standard_normal((5, 64))
    out, lse2, *_ = MD.prefill(q, kn, pe, v, [0, 3], [0, 5], 0.1, True)
    for i in range(3):
        x = 0.1 * (kn[:3 + i, 1] @ q[i, 1, :128] + pe[:3 + i] @ q[i, 1, 128:])
        assert np.isclose(lse2[i, 1], np.log2(np.exp(x).sum()))
        assert np.allclose(out[i, 1], np.exp(x) @ v[:3 + i, 1] / np.exp(x).sum())
    _, none, *_ = MD.prefill(q, kn[:1], pe[:1], v[:1], [0, 3], [0, 1], 0.1, True)
    assert np.isneginf(none[:2]).all() and np.isfinite(none[2]).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_turned_operands_keep_their_products(layout):
    """Queries and keys turned by their positions: products depend on the
    difference alone; scales are powers of two and codes use the whole range."""
    rng = np.random.default_rng(4)
    cs = RO.table(64, 32, 1e4)
    k, q = rng.standard_normal((2, 128)), rng.standard_normal((2, 3, 128))
    one = np.ones(128)
    a = IC.keys(k, one, None, 0.0, [3, 9], cs, layout, 16)
    b = IC.keys(k, one, None, 0.0, [13, 19], cs, layout, 16)
    y0, s0, w0 = IC.queries(q, np.ones((2, 3)), 0.5, [5, 6], cs, layout, 16)
    y1, s1, _ = IC.queries(q, np.ones((2, 3)), 0.5, [15, 16], cs, layout, 16)
    assert np.allclose((y0 * s0[..., None])[0] @ a[0], (y1 * s1[..., None])[0] @ b[0])
    assert np.allclose(a.mean(1)[0] * 0 + k.std(1)[0], k.std(1)[0])
    assert (np.log2(s0) % 1 == 0).all() and np.allclose(w0, 0.5 * s0)
    top = np.abs(y0).max(2)
    assert ((top <= 448) & (top > 224)).all()
    assert np.abs(KF.decode(KF.encode(y0)) - y0).max() <= 2.0 ** -4 * 448
