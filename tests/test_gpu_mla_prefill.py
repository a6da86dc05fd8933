"""GPU parity of dsa_mla_prefill with the fp64 oracle (oracle/mla_dense.py).

Bounds, from the arithmetic.  A score is a sum of 192 products in fp32: within
192 half steps of its terms' sum, 192 * 2^-24 < 2^-16 of reach; scaled and
exponentiated with 2^-22 more, so a weight is within d = 2^-16 reach + 2^-20 of
itself.  Weights enter the value product rounded to the type (u = 2^-8 or 2^-11;
in fp16 those below 2^-14 of the row's reference by at most 2^-25 of it, and the
largest weight is at least the reference's 1), the normaliser sums them in fp32;
both sums lose at most n 2^-24 <= 2^-11 of themselves for n up to 8192 keys in
any order.  So out is within (u + 2 d + 2^-10) size (+ n 2^-25 max |v| in fp16),
plus its own rounding u |out|, and lse2 within (d + 2^-11) log2 e."""
import numpy as np
import pytest
import torch

from oracle import mla_dense as MD
from tests import gpu_cases as G

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
SCALE = 192.0 ** -0.5


def inputs(lens, H, dtype, seed=0, pad=0, gain=1.0):
    """q, kv (keys and values of one projection), k_pe, cu_q, cu_k."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    Tq, Tk = sum(a for a, _ in lens) + pad, sum(b for _, b in lens) + pad
    r = lambda *s: (torch.randn(s, device="cuda", generator=g) * gain).to(dtype)   # noqa: E731
    cu = lambda ns: torch.tensor(np.concatenate([[0], np.cumsum(ns)]), dtype=torch.int32, device="cuda")  # noqa: E731
    return r(Tq, H, 192), r(Tk, H, 256), r(Tk, 64), cu([a for a, _ in lens]), cu([b for _, b in lens])


def check(q, kn, pe, v, cu_q, cu_k, scale, causal, out, lse2):
    f = lambda t: t.double().cpu().numpy()   # noqa: E731
    want, want2, size, reach = MD.prefill(f(q), f(kn), f(pe), f(v), cu_q.tolist(), cu_k.tolist(), scale, causal)
    rows = ~np.isnan(want2[:, 0]) if want2.shape[1] else np.zeros(0, bool)
    u = torch.finfo(q.dtype).eps / 2
    d = 2.0 ** -16 * reach + 2.0 ** -20
    tol = (u + 2 * d[..., None] + 2.0 ** -10) * size + u * np.abs(want) + 1e-7
    if q.dtype == torch.float16:
        tol += v.shape[0] * 2.0 ** -25 * float(torch.nan_to_num(v.float(), posinf=0, neginf=0).abs().max())
    got, got2 = f(out), f(lse2)
    assert np.array_equal(np.isneginf(got2[rows]), np.isneginf(want2[rows]))
    assert (np.abs(got[rows] - want[rows]) <= tol[rows]).all(), np.nanmax((np.abs(got - want) / tol)[rows])
    fin = np.isfinite(want2) & rows[:, None]
    assert (np.abs(got2[fin] - want2[fin]) <= (d[fin] + 2.0 ** -11) * np.log2(np.e)).all()


CASES = [
    ([(1, 1)], 1), ([(1, 1)], 3), ([(2, 1)], 2), ([(1, 129)], 2), ([(128, 128)], 1), ([(129, 129)], 2),
    ([(255, 255)], 1), ([(257, 257)], 3), ([(300, 200)], 2), ([(200, 300)], 2), ([(16, 400)], 5),
    ([(0, 7), (5, 0), (3, 3), (0, 0), (70, 130)], 2), ([(1, 1), (17, 17), (130, 131), (64, 640), (33, 5)], 4),
    ([(520, 520)], 2)]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,H", CASES)
def test_parity(lens, H, causal, kind):
    import dsa_sparse_indexer_gb300 as dsa
    q, kv, pe, cu_q, cu_k = inputs(lens, H, TYPES[kind])
    g = G.Guards()
    out, lse2 = g.empty((q.shape[0], H, 128), TYPES[kind]), g.empty((q.shape[0], H), torch.float32)
    err = dsa.new_error_flags("cuda")
    dsa.mla_prefill(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE, causal, out=out, lse2=lse2, err_flags=err)
    g.check()
    assert int(err) == 0
    check(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE, causal, out, lse2)


@pytest.mark.parametrize("causal", [True, False])
def test_many_items_a_cta(causal):
    """More (head, query block) items than SMs: barriers' phases run on across items."""
    import dsa_sparse_indexer_gb300 as dsa
    lens, H = [(40, 40), (300, 333), (1, 250), (140, 140)], 96
    q, kv, pe, cu_q, cu_k = inputs(lens, H, torch.bfloat16, seed=5)
    out, lse2 = dsa.mla_prefill(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE, causal)
    check(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE, causal, out, lse2)


@pytest.mark.parametrize("lens,H", [([(40, 9000)], 1), ([(300, 5000)], 2), ([(7, 4000), (3, 10), (9, 2049)], 1)])
def test_split_keys(lens, H):
    """Few queries, many keys: split over CTAs and joined; the same without a workspace."""
    import dsa_sparse_indexer_gb300 as dsa
    from dsa_sparse_indexer_gb300 import _lib
    q, kv, pe, cu_q, cu_k = inputs(lens, H, torch.bfloat16, seed=7)
    Tq, Tk = q.shape[0], kv.shape[0]
    assert _lib.load().dsa_mla_prefill_work(Tq, Tk, len(lens), H) > 0
    out, lse2 = dsa.mla_prefill(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE)
    check(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE, True, out, lse2)
    o1, l1 = torch.empty_like(out), torch.empty_like(lse2)
    _lib.call("dsa_mla_prefill", q.data_ptr(), q.stride(0), q.stride(1), kv.data_ptr(), kv.stride(0), 256,
              pe.data_ptr(), 64, kv[..., 128:].data_ptr(), kv.stride(0), 256, cu_q.data_ptr(), cu_k.data_ptr(),
              len(lens), Tq, Tk, H, 0, SCALE, 1, o1.data_ptr(), l1.data_ptr(), None, None,
              torch.cuda.current_stream().cuda_stream)
    check(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE, True, o1, l1)


@pytest.mark.parametrize("split", [False, True])
def test_anything_behind_the_sequences(split):
    """Rows behind the last sequence: NaN goes in, nothing comes out; between
    sequences each sees its own rows alone."""
    import dsa_sparse_indexer_gb300 as dsa
    lens, H = ([(9, 3001)], 1) if split else ([(130, 133), (20, 37)], 3)
    q, kv, pe, cu_q, cu_k = inputs(lens, H, torch.bfloat16, seed=9, pad=50)
    nq, nk = int(cu_q[-1]), int(cu_k[-1])
    q[nq:], kv[nk:], pe[nk:] = float("nan"), float("inf"), float("nan")
    out = torch.full((q.shape[0], H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse2 = torch.full((q.shape[0], H), 7.0, device="cuda")
    dsa.mla_prefill(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE, out=out, lse2=lse2)
    assert (out[nq:] == 7.0).all() and (lse2[nq:] == 7.0).all()
    check(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE, True, out, lse2)
    if not split:                                # a neighbour's NaN stays with it
        clean = out[:130].clone()
        kv[133:nk] = float("nan")
        dsa.mla_prefill(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE, out=out, lse2=lse2)
        assert torch.equal(out[:130], clean) and torch.isnan(out[130:nq]).all()


def test_masked_keys_may_hold_anything():
    """Keys (not values) that a query does not see: infinities and NaN."""
    import dsa_sparse_indexer_gb300 as dsa
    q, kv, pe, cu_q, cu_k = inputs([(40, 40)], 2, torch.bfloat16, seed=11)
    want, want2 = dsa.mla_prefill(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE)
    kv[30:35, :, :128], kv[35:, :, :128] = float("nan"), float("inf")
    out, lse2 = dsa.mla_prefill(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE)
    assert torch.equal(out[:30], want[:30]) and torch.equal(lse2[:30], want2[:30])


@pytest.mark.parametrize("scale", [0.0, -0.05, 3.0])
def test_scales_and_moving_references(scale):
    """Scores that grow along the keys make every tile's reference move."""
    import dsa_sparse_indexer_gb300 as dsa
    q, kv, pe, cu_q, cu_k = inputs([(150, 700)], 2, torch.bfloat16, seed=13)
    kv[..., :128] *= torch.linspace(3, 0.1, 700, device="cuda")[:, None, None].bfloat16()
    out, lse2 = dsa.mla_prefill(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, scale, False)
    check(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, scale, False, out, lse2)


def test_strides():
    """Queries within wider heads, keys and values of separate projections, a
    shared part within a cache row."""
    import dsa_sparse_indexer_gb300 as dsa
    q, kv, pe, cu_q, cu_k = inputs([(70, 90), (3, 200)], 3, torch.bfloat16, seed=15)
    wq = torch.zeros((q.shape[0], 5, 200), dtype=q.dtype, device="cuda")
    wq[:, 1:4, 8:] = q
    kn, v = kv[..., :128].contiguous(), kv[..., 128:].transpose(0, 1).contiguous().transpose(0, 1)
    row = torch.zeros((pe.shape[0], 576), dtype=q.dtype, device="cuda")
    row[:, 512:] = pe
    a = dsa.mla_prefill(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE)
    b = dsa.mla_prefill(wq[:, 1:4, 8:], kn, row[:, 512:], v, cu_q, cu_k, SCALE)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_bad_bounds_are_flagged_and_kept_inside():
    import dsa_sparse_indexer_gb300 as dsa
    q, kv, pe, _, _ = inputs([(40, 40)], 1, torch.bfloat16, seed=17)
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    for cu_q, cu_k in ((i(0, 41), i(0, 40)), (i(-3, 40), i(0, 40)), (i(0, 40), i(0, 99)), (i(30, 10), i(0, 40))):
        err = dsa.new_error_flags("cuda")
        dsa.mla_prefill(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE, err_flags=err)
        assert int(err) == dsa.DSA_FLAG_BOUNDS


def test_parts_of_a_context_combine():
    """A chunk's own causal part and its earlier context, merged by lse_combine."""
    import dsa_sparse_indexer_gb300 as dsa
    q, kv, pe, cu_q, cu_k = inputs([(60, 400)], 2, torch.bfloat16, seed=19)
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    out, lse2 = torch.empty((2, 60, 2, 128), dtype=q.dtype, device="cuda"), torch.empty((2, 60, 2), device="cuda")
    dsa.mla_prefill(q, kv[:340, :, :128], pe[:340], kv[:340, :, 128:], cu_q, i(0, 340), SCALE, False,
                    out=out[0], lse2=lse2[0])
    dsa.mla_prefill(q, kv[340:, :, :128], pe[340:], kv[340:, :, 128:], cu_q, i(0, 60), SCALE, True,
                    out=out[1], lse2=lse2[1])
    both, lse = dsa.lse_combine(out, lse2)
    whole, whole2 = dsa.mla_prefill(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE)
    # three roundings of the output's size and the weights' of both forms
    assert (both.float() - whole.float()).abs().max() <= 6 * 2.0 ** -8 * kv.float().abs().max()
    assert (lse / np.log(2.0) - whole2).abs().max() <= 4e-3


def test_graph_and_stream():
    import dsa_sparse_indexer_gb300 as dsa
    q, kv, pe, cu_q, cu_k = inputs([(40, 5000)], 1, torch.bfloat16, seed=21)
    args = (q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE)
    want, want2 = dsa.mla_prefill(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse2 = torch.zeros_like(want), torch.zeros_like(want2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dsa.mla_prefill(*args, out=out, lse2=lse2)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse2, want2)
    cu_k[1] = 4000                               # sizes are the device's
    graph.replay()
    torch.cuda.synchronize()
    check(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE, True, out, lse2)


def test_refusals():
    import dsa_sparse_indexer_gb300 as dsa
    q, kv, pe, cu_q, cu_k = inputs([(4, 4)], 2, torch.bfloat16)
    kn, v = kv[..., :128], kv[..., 128:]
    for bad in ((q.float(), kn, pe, v), (q, kn.half(), pe, v), (q[..., :128], kn, pe, v), (q, kn[:, :1], pe, v),
                (q, kn, pe[:, :32], v), (q, kn, pe, v[:3]), (q.cpu(), kn, pe, v), (q[0], kn, pe, v)):
        with pytest.raises((TypeError, ValueError)):
            dsa.mla_prefill(*bad, cu_q, cu_k, SCALE)
    with pytest.raises(ValueError):
        dsa.mla_prefill(q, kn, pe, v, cu_q, cu_k[:1], SCALE)
    with pytest.raises(ValueError):
        dsa.mla_prefill(q.clone().requires_grad_(), kn, pe, v, cu_q, cu_k, SCALE)
    with pytest.raises(dsa.DSAError):
        dsa.mla_prefill(q, kn, pe, v, cu_q, cu_k, float("nan"))
    odd = torch.zeros((4, 2, 193), dtype=q.dtype, device="cuda")[..., 1:]
    with pytest.raises(dsa.DSAError):
        dsa.mla_prefill(odd, kn, pe, v, cu_q, cu_k, SCALE)
    with pytest.raises(dsa.DSAError):           # heads that share their rows
        dsa.mla_prefill(q, kn[:, :1].expand(4, 2, 128), pe, v, cu_q, cu_k, SCALE)
    none = dsa.mla_prefill(q[:0], kn, pe, v, cu_q * 0, cu_k, SCALE)
    assert none[0].shape == (0, 2, 128)


def test_no_keys_and_many_sequences():
    import dsa_sparse_indexer_gb300 as dsa
    q, kv, pe, cu_q, cu_k = inputs([(5, 0), (3, 0)], 2, torch.bfloat16)
    out, lse2 = dsa.mla_prefill(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE)
    assert (out == 0).all() and torch.isneginf(lse2).all()
    lens = [((7 * i) % 11, (5 * i) % 23) for i in range(100)]
    q, kv, pe, cu_q, cu_k = inputs(lens, 2, torch.bfloat16, seed=23)
    out, lse2 = dsa.mla_prefill(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE)
    check(q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE, True, out, lse2)


def test_offsets_past_32_bits():
    """Keys and values whose elements lie past 2^31 of their tensors."""
    import dsa_sparse_indexer_gb300 as dsa
    far, H = 66000, 128
    kv = torch.empty((far + 40, H, 256), dtype=torch.bfloat16, device="cuda")
    q, near, pe, _, _ = inputs([(5, 40)], H, torch.bfloat16, seed=25)
    kv[far:] = near
    pes = torch.empty((far + 40, 64), dtype=torch.bfloat16, device="cuda")
    pes[far:] = pe
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    a = dsa.mla_prefill(q, kv[..., :128], pes, kv[..., 128:], i(0, 0, 5), i(0, far, far + 40), SCALE)
    b = dsa.mla_prefill(q, near[..., :128], pe, near[..., 128:], i(0, 5), i(0, 40), SCALE)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_streams_and_the_same_twice():
    """Two calls at once, each with its own outputs and workspace, give what one gives."""
    import dsa_sparse_indexer_gb300 as dsa
    q, kv, pe, cu_q, cu_k = inputs([(40, 3000), (513, 700)], 2, torch.bfloat16, seed=27)
    args = (q, kv[..., :128], pe, kv[..., 128:], cu_q, cu_k, SCALE)
    want = dsa.mla_prefill(*args)
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got.append(dsa.mla_prefill(*args))
    torch.cuda.synchronize()
    assert all(torch.equal(g[0], want[0]) and torch.equal(g[1], want[1]) for g in got)


@pytest.mark.parametrize("n", [33, 128, 129])
def test_sequences_in_any_order(n):
    """Sequences are taken longest first, up to 128 of them: lengths with repeats,
    none ascending or descending, some empty."""
    rng = np.random.default_rng(n)
    lens = [(int(a), int(b)) for a, b in zip(rng.integers(0, 3, n), rng.integers(0, 200, n))]
    lens[n // 2] = (40, 300)
    import dsa_sparse_indexer_gb300 as dsa
    q, kv, pe, cu_q, cu_k = inputs(lens, 2, torch.bfloat16, seed=n)
    kn, v = kv[..., :128], kv[..., 128:]
    err = dsa.new_error_flags("cuda")
    out, lse2 = dsa.mla_prefill(q, kn, pe, v, cu_q, cu_k, SCALE, err_flags=err)
    assert int(err) == 0
    check(q, kn, pe, v, cu_q, cu_k, SCALE, True, out, lse2)
