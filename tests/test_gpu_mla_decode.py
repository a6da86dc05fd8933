"""GPU parity of dsa_mla_decode with the fp64 oracle (oracle/mla_dense.py).

Bounds as for the expanded form (a score sums 576 products: 576 * 2^-24 < 2^-14
of reach; n at most 8192): out within (2^-8 + 2 d + 2^-10) size + 2^-8 |out|,
lse2 within (d + 2^-11) log2 e, d = 2^-14 reach + 2^-20."""
import numpy as np
import pytest
import torch

from oracle import mla_dense as MD
from tests import gpu_cases as G

pytestmark = pytest.mark.gpu
SCALE = 192.0 ** -0.5


def inputs(drafts, lens, H, S=1, I=1, block=64, seed=0, spare=0, cols=None):
    rng = np.random.default_rng(seed)
    reqs = len(lens)
    local0 = [-(-n // S) + I for n in lens]
    cols = cols or max(1, -(-max(local0) // block))
    table = np.stack([rng.permutation(reqs * cols).reshape(reqs, cols) for _ in range(S)]).astype(np.int32)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rows = sum(drafts) + spare
    q = torch.randn((rows, H, 576), device="cuda", generator=g).bfloat16()
    cache = torch.randn((S, reqs * cols * block, 576), device="cuda", generator=g).bfloat16()
    starts = torch.tensor(np.concatenate([[0], np.cumsum(drafts)]), dtype=torch.int32, device="cuda")
    return (q, cache, torch.from_numpy(table).cuda(), block, starts,
            torch.tensor(lens, dtype=torch.int32, device="cuda"), I)


def tree(drafts, spare=0, words=None, seed=0):
    """Every draft's parent is one of those before it, or none."""
    rng = np.random.default_rng(seed)
    words = words or -(-max(max(drafts), 1) // 32)
    bits = np.zeros((sum(drafts) + spare, words * 32), bool)
    at = 0
    for n in drafts:
        for j in range(n):
            p = rng.integers(-1, j) if j else -1
            if p >= 0:
                bits[at + j] = bits[at + p]
            if j < words * 32:
                bits[at + j, j] = True
        at += n
    w = (bits.reshape(len(bits), words, 32).astype(np.int64) << np.arange(32)).sum(-1)
    return torch.from_numpy(np.where(w >= 1 << 31, w - (1 << 32), w).astype(np.int32)).cuda()


def check(args, scale, mask, out, lse2):
    q, cache, table, block, starts, lens, I = args
    f = lambda t: t.double().cpu().numpy()   # noqa: E731
    want, want2, size, reach = MD.decode(f(q), f(cache), table.cpu().numpy(), block, starts.tolist(), lens.tolist(),
                                         cache.shape[0], I, scale, None if mask is None else mask.cpu().numpy())
    rows = ~np.isnan(want2)
    d = 2.0 ** -14 * reach + 2.0 ** -20
    tol = (2.0 ** -8 + 2 * d[..., None] + 2.0 ** -10) * size + 2.0 ** -8 * np.abs(want) + 1e-7
    got, got2 = f(out), f(lse2)
    assert np.array_equal(np.isneginf(got2[rows]), np.isneginf(want2[rows]))
    assert (np.abs(got[rows] - want[rows]) <= tol[rows]).all(), (np.abs(got - want) / tol)[rows].max()
    fin = np.isfinite(want2)
    assert (np.abs(got2[fin] - want2[fin]) <= (d[fin] + 2.0 ** -11) * np.log2(np.e)).all()


CASES = [
    # drafts, lens, H, S, I, block, tree
    ([1], [1], 1, 1, 1, 64, False), ([1], [127], 16, 1, 1, 16, False), ([1, 1], [129, 5], 8, 2, 1, 32, False),
    ([1, 1, 1], [300, 1, 77], 16, 4, 2, 64, False), ([5], [5], 3, 1, 1, 64, False), ([7, 1], [260, 64], 16, 2, 4, 64, False),
    ([4], [3], 2, 1, 1, 64, False), ([0, 2, 0], [9, 2, 0], 4, 2, 1, 64, False), ([3], [200], 40, 1, 1, 128, True),
    ([8, 3], [140, 3], 16, 2, 1, 64, True), ([33], [33], 2, 1, 1, 64, True), ([40, 2], [170, 259], 3, 3, 16, 192, True),
    ([2], [700], 64, 1, 1, 64, False)]


@pytest.mark.parametrize("drafts,lens,H,S,I,block,with_tree", CASES)
def test_parity(drafts, lens, H, S, I, block, with_tree):
    import dsa_sparse_indexer_gb300 as dsa
    args = inputs(drafts, lens, H, S, I, block, seed=len(lens) * 7 + H)
    mask = tree(drafts) if with_tree else None
    rows = args[0].shape[0]
    g = G.Guards()
    out, lse2 = g.empty((S, rows, H, 512), torch.bfloat16), g.empty((S, rows, H), torch.float32)
    err = dsa.new_error_flags("cuda")
    dsa.mla_decode(*args, SCALE, tree_mask=mask, out=out, lse2=lse2, err_flags=err)
    g.check()
    assert int(err) == 0
    check(args, SCALE, mask, out, lse2)


PAIRS = [
    ([1, 2], [200, 131], 128, 1, 1, 64, False), ([3], [390], 64, 2, 1, 64, False), ([8, 5, 8], [150, 300, 8], 32, 2, 4, 32, True),
    ([61], [130], 8, 1, 1, 16, True), ([2, 1], [60, 61], 192, 1, 1, 64, False), ([20], [20], 20, 4, 1, 64, True)]


@pytest.mark.parametrize("drafts,lens,H,S,I,block,with_tree", PAIRS)
def test_parity_of_pairs_of_ctas(drafts, lens, H, S, I, block, with_tree):
    test_parity(drafts, lens, H, S, I, block, with_tree)


@pytest.mark.parametrize("H,drafts", [(4, 1), (64, 3)])
def test_many_items_a_cta(H, drafts):
    """More items than CTAs: barriers' phases run on across items; empty shards between."""
    import dsa_sparse_indexer_gb300 as dsa
    lens = [3 + 29 * i % 260 for i in range(60)]
    args = inputs([min(drafts, n) for n in lens], lens, H, 4, 2, 64, seed=3)
    out, lse2 = dsa.mla_decode(*args, SCALE)
    check(args, SCALE, None, out, lse2)


@pytest.mark.parametrize("H,drafts", [(2, [1]), (100, [2]), (3, [1, 4])])
def test_split_tokens(H, drafts):
    """Few rows, many tokens: split over CTAs and joined; the same without a workspace."""
    import dsa_sparse_indexer_gb300 as dsa
    from dsa_sparse_indexer_gb300 import _lib
    lens = [4000, 1300][:len(drafts)]
    args = inputs(drafts, lens, H, 1, 1, 64, seed=5)
    q, cache, table, block, starts, ln, I = args
    rows = q.shape[0]
    assert _lib.load().dsa_mla_decode_work(rows, 1, H, len(lens), table.shape[2], block) > 0
    out, lse2 = dsa.mla_decode(*args, SCALE)
    check(args, SCALE, None, out, lse2)
    o1, l1 = torch.empty_like(out), torch.empty_like(lse2)
    _lib.call("dsa_mla_decode", q.data_ptr(), cache.data_ptr(), cache.shape[1], table.data_ptr(), len(lens),
              table.shape[2], block, starts.data_ptr(), ln.data_ptr(), None, 0, rows, 1, I, H, SCALE, o1.data_ptr(),
              l1.data_ptr(), None, None, torch.cuda.current_stream().cuda_stream)
    check(args, SCALE, None, o1, l1)


@pytest.mark.parametrize("H,drafts", [(16, 2), (96, 2)])
def test_anything_behind_the_tokens(H, drafts):
    """Stale slots behind a sequence's last token hold NaN and infinities."""
    import dsa_sparse_indexer_gb300 as dsa
    args = inputs([drafts] * 3, [100, 130, 66], H, 2, 1, 64, seed=7)
    q, cache, table, block, starts, lens, I = args
    want = dsa.mla_decode(*args, SCALE)
    used = torch.zeros(cache.shape[:2], dtype=torch.bool, device="cuda")
    for r, n in enumerate(lens.tolist()):
        for s in range(2):
            loc = torch.arange((n - s + 1) // 2, device="cuda")
            used[s, table[s, r].long()[loc // block] * block + loc % block] = True
    cache[~used] = float("nan")
    got = dsa.mla_decode(*args, SCALE)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    cache[~used] = float("inf")
    got = dsa.mla_decode(*args, SCALE)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("H", [16, 128])
def test_rows_behind_the_last_request(H):
    import dsa_sparse_indexer_gb300 as dsa
    args = inputs([2, 1], [90, 30], H, 1, 1, 64, seed=9, spare=5)
    out = torch.full((1, 8, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse2 = torch.full((1, 8, H), 7.0, device="cuda")
    args[0][3:] = float("nan")
    dsa.mla_decode(*args, SCALE, out=out, lse2=lse2)
    assert (out[:, 3:] == 7.0).all() and (lse2[:, 3:] == 7.0).all()
    check(args, SCALE, None, out, lse2)


def test_empty_mask_rows_and_bits_past_the_words():
    import dsa_sparse_indexer_gb300 as dsa
    args = inputs([40], [40], 4, 1, 1, 64, seed=11)
    mask = torch.zeros((40, 1), dtype=torch.int32, device="cuda")
    mask[39, 0] = -2 ** 31
    out, lse2 = dsa.mla_decode(*args, SCALE, tree_mask=mask)
    assert torch.isneginf(lse2[0, :39]).all() and (out[0, :39] == 0).all()
    check(args, SCALE, mask, out, lse2)


@pytest.mark.parametrize("H", [16, 128])
def test_bad_pages_and_lengths(H):
    """Entries outside the cache leave their tokens out; lengths past the table are cut."""
    import dsa_sparse_indexer_gb300 as dsa
    args = inputs([2, 1], [260, 200], H, 1, 1, 64, seed=13)
    args[2][0, 0, 1], args[2][0, 1, 0], args[2][0, 0, 4] = -5, 2 ** 31 - 1, 2 ** 25
    err = dsa.new_error_flags("cuda")
    out, lse2 = dsa.mla_decode(*args, SCALE, err_flags=err)
    assert int(err) == dsa.DSA_FLAG_BOUNDS
    check(args, SCALE, None, out, lse2)
    args = inputs([2, 1], [100, 50], H, 1, 1, 64, seed=14)
    args[5][0], args[5][1] = 129 + 64, -4
    err = dsa.new_error_flags("cuda")
    out, lse2 = dsa.mla_decode(*args, SCALE, err_flags=err)
    assert int(err) == dsa.DSA_FLAG_BOUNDS and torch.isneginf(lse2[0, 2]).all()
    check(args, SCALE, None, out, lse2)
    for starts in ((0, 4, 3), (-1, 1, 3), (2, 1, 3)):
        args[4].copy_(torch.tensor(starts, dtype=torch.int32))
        err = dsa.new_error_flags("cuda")
        dsa.mla_decode(*args, SCALE, err_flags=err)
        assert int(err) == dsa.DSA_FLAG_BOUNDS


@pytest.mark.parametrize("scale", [0.0, -0.05, 2.0])
@pytest.mark.parametrize("H", [16, 128])
def test_scales_and_moving_references(scale, H):
    import dsa_sparse_indexer_gb300 as dsa
    args = inputs([2], [600], H, 1, 1, 64, seed=15)
    table = args[2][0, 0].long()
    loc = torch.arange(600, device="cuda")
    args[1][0, table[loc // 64] * 64 + loc % 64] *= torch.linspace(3, 0.1, 600, device="cuda")[:, None].bfloat16()
    out, lse2 = dsa.mla_decode(*args, scale)
    check(args, scale, None, out, lse2)


def test_all_tokens_selected_is_the_sparse_attention():
    """Beside sparse_mla_decode over every slot, and combined over shards."""
    import dsa_sparse_indexer_gb300 as dsa
    args = inputs([1, 1], [300, 170], 128, 2, 1, 64, seed=17)
    q, cache, table, block, starts, lens, I = args
    out, lse2 = dsa.mla_decode(*args, SCALE)
    K = 192
    slots = torch.full((2, 2, K), -1, dtype=torch.int32, device="cuda")
    counts = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    for r, n in enumerate(lens.tolist()):
        for s in range(2):
            loc = torch.arange((n - s + 1) // 2, device="cuda")
            slots[s, r, :loc.numel()] = (table[s, r].long()[loc // block] * block + loc % block).int()
            counts[s, r] = loc.numel()
    o2, l2 = dsa.sparse_mla_decode(q, cache, slots, counts, SCALE)
    assert (lse2 - l2).abs().max() <= 2e-3
    # both round weights (2^-8) and outputs (2^-8) of values up to the largest
    assert (out.float() - o2.float()).abs().max() <= 4 * 2.0 ** -8 * cache.float().abs().max()
    dsa.lse_combine(out, lse2)


@pytest.mark.parametrize("H,drafts", [(2, 1), (128, 2)])
def test_graph_and_stream(H, drafts):
    import dsa_sparse_indexer_gb300 as dsa
    args = inputs([drafts], [3000], H, 1, 1, 64, seed=19)
    want, want2 = dsa.mla_decode(*args, SCALE)
    out, lse2 = torch.zeros_like(want), torch.zeros_like(want2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.mla_decode(*args, SCALE, out=out, lse2=lse2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse2, want2)
    args[5][0] = 2500                            # lengths are the device's
    graph.replay()
    torch.cuda.synchronize()
    check(args, SCALE, None, out, lse2)


def test_refusals():
    import dsa_sparse_indexer_gb300 as dsa
    args = inputs([1], [10], 4)
    q, cache, table, block, starts, lens, I = args
    for bad in ((q.half(), cache, table, block, starts, lens, I), (q[..., :512], cache, table, block, starts, lens, I),
                (q, cache[..., :512], table, block, starts, lens, I), (q, cache, table.long(), block, starts, lens, I),
                (q, cache, table, block, starts[:1], lens, I), (q, cache, table[:, :, 0], block, starts, lens, I),
                (q.cpu(), cache, table, block, starts, lens, I)):
        with pytest.raises((TypeError, ValueError)):
            dsa.mla_decode(*bad, SCALE)
    for bad in ((q, cache, table, 48, starts, lens, I), (q, cache, table, block, starts, lens, 0),
                (q, cache, table, 0, starts, lens, I)):
        with pytest.raises(dsa.DSAError):
            dsa.mla_decode(*bad, SCALE)
    with pytest.raises(ValueError):
        dsa.mla_decode(*args, SCALE, tree_mask=torch.zeros((2, 1), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        dsa.mla_decode(q.clone().requires_grad_(), *args[1:], SCALE)
    with pytest.raises(dsa.DSAError):
        dsa.mla_decode(*args, float("inf"))
    none = dsa.mla_decode(q[:0], cache, table, block, starts * 0, lens, I, SCALE)
    assert none[0].shape == (1, 0, 4, 512)


@pytest.mark.parametrize("H,drafts", [(16, 1), (128, 1), (128, 2)])
def test_offsets_past_32_bits(H, drafts):
    """Pages whose rows lie past 2^31 elements of a shard's cache, and of the cache."""
    import dsa_sparse_indexer_gb300 as dsa
    n_slots = 64 * 60000
    cache = torch.empty((2, n_slots, 576), dtype=torch.bfloat16, device="cuda")
    args = inputs([drafts], [150], H, 2, 1, 64, seed=21)
    q, near, table, block, starts, lens, I = args
    far = table + (60000 - int(table.max()) - 1)
    for s in range(2):
        for p in table[s, 0].tolist():
            at = (p + 60000 - int(table.max()) - 1) * 64
            cache[s, at:at + 64] = near[s, p * 64:p * 64 + 64]
    a = dsa.mla_decode(q, cache, far.contiguous(), block, starts, lens, I, SCALE)
    b = dsa.mla_decode(*args, SCALE)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("H,drafts", [(2, [1]), (128, [5, 3])])
def test_two_streams_and_the_same_twice(H, drafts):
    """Two calls at once, each with its own outputs and workspace, give what one gives."""
    import dsa_sparse_indexer_gb300 as dsa
    args = inputs(drafts, [2500, 900][:len(drafts)], H, 2, 1, 64, seed=23)
    want = dsa.mla_decode(*args, SCALE)
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got.append(dsa.mla_decode(*args, SCALE))
    torch.cuda.synchronize()
    assert all(torch.equal(g[0], want[0]) and torch.equal(g[1], want[1]) for g in got)


def test_split_tree():
    """A tree over few rows: its drafts lie in the last of the parts."""
    import dsa_sparse_indexer_gb300 as dsa
    from dsa_sparse_indexer_gb300 import _lib
    args = inputs([33], [3000], 4, 2, 4, 64, seed=25)
    mask = tree([33], seed=25)
    assert _lib.load().dsa_mla_decode_work(33, 2, 4, 1, args[2].shape[2], 64) > 0
    out, lse2 = dsa.mla_decode(*args, SCALE, tree_mask=mask)
    check(args, SCALE, mask, out, lse2)


@pytest.mark.parametrize("reqs,H", [(33, 40), (128, 2), (129, 2)])
def test_requests_in_any_order(reqs, H):
    """Requests are taken longest first, up to 128 of them: lengths with repeats,
    none ascending or descending, some empty."""
    import dsa_sparse_indexer_gb300 as dsa
    rng = np.random.default_rng(reqs)
    drafts = [int(x) for x in rng.integers(0, 3, reqs)]
    lens = [int(x) for x in rng.integers(0, 200, reqs)]
    args = inputs(drafts, lens, H, 2, 1, 16, seed=reqs)
    err = dsa.new_error_flags("cuda")
    out, lse2 = dsa.mla_decode(*args, SCALE, err_flags=err)
    assert int(err) == 0
    check(args, SCALE, None, out, lse2)


UNEVEN = [([20, 1, 0, 1, 1, 1], [300, 5, 9, 1, 140, 128], 4, 16), ([30, 1, 1, 1], [31, 700, 129, 64], 3, 64),
          ([1, 70, 1, 1, 1, 1, 1, 1], [900, 70, 1, 2, 300, 17, 128, 256], 2, 32)]


@pytest.mark.parametrize("with_tree", [False, True])
@pytest.mark.parametrize("drafts,lens,H,block", UNEVEN)
def test_few_rows_and_one_request_of_many(drafts, lens, H, block, with_tree):
    """Few rows a request on average, one with several blocks of them."""
    test_parity(drafts, lens, H, 2, 1, block, with_tree)


def test_split_tokens_of_32_rows():
    """Two tokens of 16 heads and one of 32, many tokens in parts."""
    import dsa_sparse_indexer_gb300 as dsa
    from dsa_sparse_indexer_gb300 import _lib
    for H, drafts in ((16, [2]), (32, [1])):
        args = inputs(drafts, [5000], H, 1, 1, 64, seed=H)
        rows, table = args[0].shape[0], args[2]
        need = _lib.load().dsa_mla_decode_work(rows, 1, H, 1, table.shape[2], 64)
        assert need > 0
        out, lse2 = dsa.mla_decode(*args, SCALE)
        check(args, SCALE, None, out, lse2)
