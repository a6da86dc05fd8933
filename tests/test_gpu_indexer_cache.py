"""GPU parity of dsa_indexer_key_insert and dsa_indexer_query_fp8 with the fp64
oracle (oracle/indexer_cache.py).

Bounds: a code is its exact value rounded once, except where fp32 arithmetic
puts it on the other side of a rounding border: code value within half a step
(2^-4 of the value, 2^-10 below 2^-6) plus e, the fp32 error.  For keys, layer
norm over 128 values: the mean and the variance sum 128 terms (2^-17 of their
size), a few more roundings: e = 2^-15 (|y| + the normed values' largest times
|weight| + |bias|).  For queries the rotation alone: e = 2^-22 of the head's
largest.  Scales and weights follow the exact values: weights within 2^-22."""
import numpy as np
import pytest
import torch

from oracle import indexer_cache as IC
from oracle import indexer_logits as IL
from oracle import kv_fp8 as KF
from oracle import rope as RO

pytestmark = pytest.mark.gpu

TURNS = [("half", 64, 0), ("interleaved", 64, 0), ("half", 128, 0), ("interleaved", 2, 126), ("half", 6, 5),
         ("interleaved", 50, 33), ("half", 64, 64)]


def half_step(y):
    return np.where(np.abs(y) < 2.0 ** -6, 2.0 ** -10, 2.0 ** -4 * np.abs(y))


def cos_sin(rot, max_pos=300):
    return torch.from_numpy(RO.table(max_pos, rot, 1e4).astype(np.float32)).cuda()


@pytest.mark.parametrize("layout,rot,first", TURNS)
@pytest.mark.parametrize("T,S,bias", [(1, 1, True), (7, 4, False), (300, 2, True), (50, 20, False)])
def test_keys(T, S, bias, layout, rot, first):
    import dsa_sparse_indexer_gb300 as dsa
    g = torch.Generator(device="cuda")
    g.manual_seed(T + rot)
    r = lambda *s: torch.randn(s, device="cuda", generator=g)   # noqa: E731
    wide = (r(T, 200) * 3 + 0.5).bfloat16()
    k = wide[:, 8:136]
    w, b = 1 + 0.3 * r(128), (0.2 * r(128) if bias else None)
    cs = cos_sin(rot)
    pos = torch.randint(0, 300, (T,), device="cuda", generator=g, dtype=torch.int32)
    n_slots = 2 * T + 3
    owner = torch.randint(-1, S, (T,), device="cuda", generator=g)
    slot = torch.stack([torch.randperm(n_slots, device="cuda", generator=g)[:T] for _ in range(S)])
    slots = torch.where(owner == torch.arange(S, device="cuda")[:, None], slot, -1).int()
    cache = torch.full((S, n_slots, 128), 0x11, dtype=torch.uint8, device="cuda")
    err = dsa.new_error_flags("cuda")
    got = dsa.indexer_key_insert(k, w, b, 1e-6, pos, cs, slots, cache, layout=layout, first=first, err_flags=err)
    assert got is cache and int(err) == 0
    f = lambda t: None if t is None else t.double().cpu().numpy()   # noqa: E731
    y = IC.keys(f(k), f(w), f(b), 1e-6, pos.cpu().numpy(), f(cs), layout, first)
    x = f(k) - f(k).mean(1, keepdims=True)
    top = (np.abs(x) / np.sqrt((x * x).mean(1, keepdims=True) + 1e-6)).max(1, keepdims=True)
    e = 2.0 ** -15 * (np.abs(y) + top * np.abs(f(w)).max() + (np.abs(f(b)).max() if bias else 0))
    codes, sl = cache.cpu().numpy(), slots.cpu().numpy()
    hit = np.zeros((S, n_slots), bool)
    for s in range(S):
        for t in np.nonzero(sl[s] >= 0)[0]:
            hit[s, sl[s, t]] = True
            assert (np.abs(KF.decode(codes[s, sl[s, t]]) - y[t]) <= half_step(y[t]) + e[t]).all()
    assert (codes[~hit] == 0x11).all()


def test_keys_that_saturate_and_are_not_finite():
    import dsa_sparse_indexer_gb300 as dsa
    k = torch.zeros((3, 128), dtype=torch.bfloat16, device="cuda")
    k[0, 0], k[1, 5] = 100.0, float("nan")
    w = torch.full((128,), 1e4, device="cuda")
    cache = torch.zeros((1, 4, 128), dtype=torch.uint8, device="cuda")
    z = torch.zeros(3, dtype=torch.int32, device="cuda")
    dsa.indexer_key_insert(k, w, None, 0.0, z, cos_sin(64), torch.tensor([[0, 1, 3]], dtype=torch.int32, device="cuda"),
                           cache, first=64)
    v = KF.decode(cache.cpu().numpy()[0])
    assert v[0, 0] == 448.0 and (v[0, 1:64] == -448.0).all() and np.isnan(v[1]).all()
    assert np.isnan(v[3]).all()                  # a key of equal values has no variance, and eps is 0


def test_key_positions_and_slots_out_of_range():
    import dsa_sparse_indexer_gb300 as dsa
    k = torch.randn((4, 128), device="cuda").bfloat16()
    w = torch.ones(128, device="cuda")
    cs = cos_sin(64)
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    cache = torch.zeros((1, 4, 128), dtype=torch.uint8, device="cuda")
    err = dsa.new_error_flags("cuda")
    dsa.indexer_key_insert(k, w, None, 1e-6, i(0, 0, 0, 0), cs, i(0, 1, 2, 4)[None], cache, err_flags=err)
    assert int(err) == dsa.DSA_FLAG_BOUNDS and (cache[0, 3] == 0).all()
    plain = cache.clone()                        # position 0 turns by nothing
    err = dsa.new_error_flags("cuda")
    dsa.indexer_key_insert(k, w, None, 1e-6, i(-1, 300, 0, 0), cs, i(0, 1, 2, -1)[None], cache, err_flags=err)
    assert int(err) == dsa.DSA_FLAG_BOUNDS and torch.equal(cache, plain)


@pytest.mark.parametrize("layout,rot,first", TURNS)
@pytest.mark.parametrize("T,H", [(1, 1), (3, 64), (65, 33)])
def test_queries(T, H, layout, rot, first):
    import dsa_sparse_indexer_gb300 as dsa
    g = torch.Generator(device="cuda")
    g.manual_seed(T + rot)
    q = torch.randn((T, H + 1, 144), device="cuda", generator=g)
    q = (q * torch.exp2(8 * torch.randn((T, H + 1, 1), device="cuda", generator=g))).bfloat16()[:, 1:, 8:136]
    w = torch.randn((T, H), device="cuda", generator=g)
    cs = cos_sin(rot)
    pos = torch.randint(0, 300, (T,), device="cuda", generator=g, dtype=torch.int32)
    q[0, 0] = 0.0
    got, got_w = dsa.indexer_query_fp8(q, w, pos, cs, factor=0.125, layout=layout, first=first)
    f = lambda t: t.double().cpu().numpy()   # noqa: E731
    y, scale, want_w = IC.queries(f(q), f(w), 0.125, pos.cpu().numpy(), f(cs), layout, first)
    v = KF.decode(got.cpu().numpy())
    e = 2.0 ** -22 * np.abs(y).max(2, keepdims=True)
    assert (np.abs(v - y) <= half_step(y) + e).all()
    assert (np.abs(f(got_w) - want_w) <= 2.0 ** -22 * np.abs(want_w)).all()


def test_query_scales_at_borders():
    """Largest values on, next to and far from a power of two times 448; tiny and
    infinite ones."""
    import dsa_sparse_indexer_gb300 as dsa
    tops = [448.0, 450.0, 446.0, 1.75, 1.7578125, 2.0 ** -130, 3e38, float("inf"), float("nan"), 0.0]
    q = torch.zeros((1, len(tops), 128), device="cuda")
    q[0, :, 100] = torch.tensor(tops, device="cuda")
    q[0, :, 101] = 1.0
    q[0, 5, 101] = 0.0
    q = q.bfloat16()
    w = torch.ones((1, len(tops)), device="cuda")
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, got_w = dsa.indexer_query_fp8(q, w, z, cos_sin(64))
    with np.errstate(invalid="ignore"):
        y, scale, want_w = IC.queries(q.double().cpu().numpy(), np.ones((1, len(tops))), 1.0, [0],
                                      RO.table(1, 64, 1e4), "half", 0)
    assert np.array_equal(got_w.double().cpu().numpy(), want_w)
    assert np.array_equal(got.cpu().numpy(), KF.encode(y))


def test_operands_of_the_logits():
    """Keys and queries made here, scored by indexer_logits: the oracle's logits of
    the same 8-bit values, and close to those of the exact ones."""
    import dsa_sparse_indexer_gb300 as dsa
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    T, S, I, b = 130, 2, 1, 16
    r = lambda *s: torch.randn(s, device="cuda", generator=g)   # noqa: E731
    cs = dsa.rope_table(T, 64)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    table = torch.stack([torch.randperm(8, device="cuda", generator=g) for _ in range(S)]).int().view(S, 1, 8)
    slots = dsa.slot_mapping(pos, table, b, I, token_req=torch.zeros_like(pos))
    k, w = r(T, 128).bfloat16(), torch.ones(128, device="cuda")
    cache = torch.zeros((S, 8 * b, 128), dtype=torch.uint8, device="cuda")
    dsa.indexer_key_insert(k, w, None, 1e-6, pos, cs, slots, cache)
    q, hw = r(4, 64, 128).bfloat16(), r(4, 64).abs()
    at = pos[-4:].contiguous()
    q8, w8 = dsa.indexer_query_fp8(q, hw, at, cs, factor=64.0 ** -0.5 * 128.0 ** -0.5)
    ends = at + 1
    logits = torch.zeros((S, 4, 72), device="cuda")
    dsa.indexer_logits(q8, w8, cache, table, b, ends, I, 72, row_to_req=torch.zeros_like(ends), out=logits)
    n = lambda t: t.cpu().numpy()   # noqa: E731
    a = (n(q8), n(w8), n(cache), np.zeros(4, np.int32), n(ends), S, I, n(table), b)
    want = IL.shard_logits(*a, ld=72, row_to_req=np.zeros(4, np.int32))
    mag = IL.magnitude(*a, ld=72, row_to_req=np.zeros(4, np.int32))
    inside = ~np.isnan(want)
    assert (np.abs(n(logits).astype(np.float64)[inside] - want[inside]) <= 2.0 ** -13 * mag[inside] + 1e-6).all()
    f = lambda t: t.double().cpu().numpy()   # noqa: E731
    y = IC.keys(f(k), np.ones(128), None, 1e-6, n(pos), f(cs), "half", 0)
    yq, sc, wf = IC.queries(f(q), f(hw), 64.0 ** -0.5 * 128.0 ** -0.5, n(at), f(cs), "half", 0)
    exact = (wf[:, :, None] * np.maximum(0.0, yq @ y.T)).sum(1)
    for i in range(4):
        for s in range(S):
            mine = np.arange(T)[np.arange(T) % S == s]
            mine = mine[mine < int(ends[i])]
            size = (np.abs(wf[i])[:, None] * (np.abs(yq[i]) @ np.abs(y[mine]).T)).sum(0)
            assert (np.abs(n(logits)[s, i, :mine.size] - exact[i, mine]) <= 2.0 ** -2.9 * size).all()


def test_refusals():
    import dsa_sparse_indexer_gb300 as dsa
    k = torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    w, cs = torch.ones(128, device="cuda"), cos_sin(64)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    slots, cache = pos[None].clone(), torch.zeros((1, 4, 128), dtype=torch.uint8, device="cuda")
    key = lambda **kw: dsa.indexer_key_insert(**{**dict(   # noqa: E731
        k=k, norm_weight=w, norm_bias=None, eps=1e-6, positions=pos, cos_sin_cache=cs, slot_mapping=slots,
        k_cache=cache), **kw})
    for bad in (dict(k=k.float()), dict(k=k[:, :64]), dict(norm_weight=w[:64]), dict(norm_bias=w.half()),
                dict(positions=pos.long()), dict(slot_mapping=slots[:, :1]), dict(k_cache=cache[0]),
                dict(layout="other"), dict(k_cache=cache.cpu()), dict(norm_weight=w.clone().requires_grad_())):
        with pytest.raises((TypeError, ValueError)):
            key(**bad)
    for bad in (dict(first=65), dict(first=-1), dict(eps=-1.0), dict(eps=float("nan")),
                dict(k=torch.zeros((2, 129), dtype=k.dtype, device="cuda")[:, 1:])):
        with pytest.raises(dsa.DSAError):
            key(**bad)
    q, hw = torch.zeros((2, 3, 128), dtype=torch.bfloat16, device="cuda"), torch.ones((2, 3), device="cuda")
    qry = lambda **kw: dsa.indexer_query_fp8(**{**dict(   # noqa: E731
        q=q, weights=hw, positions=pos, cos_sin_cache=cs), **kw})
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(weights=hw[:1]), dict(positions=pos[:1]), dict(layout=None),
                dict(q_out=torch.zeros((2, 3, 64), dtype=torch.uint8, device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            qry(**bad)
    for bad in (dict(first=65), dict(factor=float("inf")), dict(q=q[..., :1].expand(2, 3, 128).transpose(1, 2)[:, :3])):
        with pytest.raises((dsa.DSAError, ValueError)):
            qry(**bad)
    assert qry(q=q[:0], weights=hw[:0], positions=pos[:0])[0].shape == (0, 3, 128)
