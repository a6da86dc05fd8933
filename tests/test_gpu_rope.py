"""GPU parity of dsa_rope_table and dsa_rotary_embed with the fp64 oracle
(oracle/rope.py).

Tolerances, from the arithmetic.  Table: the angle is exact to 2^-32 turns and
p 2^-65 turns for the rounded step (together below 2^-30 turns for p < 2^31),
then rounded to fp32 as a fraction of half a turn (2^-25 pi), its cosine and
sine within 2 fp32 steps (2^-22), one product with the amplitude (2^-24): below
4e-7 of the amplitude.  Rotation: y s rounded, then x c - y s rounded:
2^-24 (|y s| + |x c - y s|) <= 2^-23 (|x| + |y|) for |c|, |s| <= 1, then one
rounding to the output's type (half a step, plus half the smallest fp16
subnormal, 2^-25)."""
import numpy as np
import pytest
import torch

from oracle import rope as RO
from tests import gpu_cases as G

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.mark.parametrize("max_pos,rot,base,scaling,factor", [
    (1, 2, 10000.0, "ntk", 4.0), (1, 256, 1e6, None, 1.0), (63, 6, 10000.0, "linear", 2.5),
    (65, 64, 10000.0, "yarn", 40.0), (1000, 96, 500000.0, "ntk", 8.0),
    (4096, 128, 500000.0, "yarn", 1.0), (262147, 64, 10000.0, "yarn", 32.0),
    (70001, 62, 10000.0, "linear", 4.0), (40003, 8, 10000.0, None, 1.0)])
def test_table(max_pos, rot, base, scaling, factor):
    import dsa_sparse_indexer_gb300 as dsa
    g = G.Guards()
    out = g.empty((max_pos, rot), torch.float32)
    got = dsa.rope_table(max_pos, rot, base, scaling, factor, amplitude=1.25, out=out)
    g.check()
    assert got is out
    want = RO.table(max_pos, rot, base, 1.25, scaling=scaling, factor=factor)
    assert np.abs(out.cpu().numpy() - want).max() <= 4e-7 * 1.25


def test_table_without_alignment():
    import dsa_sparse_indexer_gb300 as dsa
    held = torch.full((50 * 64 + 2,), 7.0, device="cuda")
    got = dsa.rope_table(50, 64, out=held[1:-1].view(50, 64))
    assert torch.equal(got, dsa.rope_table(50, 64))
    assert float(held[0]) == 7.0 and float(held[-1]) == 7.0


def _check(x, pos, cs, got, layout, first, inverse, dtype):
    xd = x.double().cpu().numpy()
    want = RO.rotate(xd, pos, cs.astype(np.float64), layout, first, inverse)
    n = cs.shape[1]
    r = np.abs(xd[..., first:first + n])
    mate = (r.reshape(*r.shape[:-1], -1, 2)[..., ::-1].reshape(r.shape) if layout == "interleaved"
            else np.roll(r, n // 2, axis=-1))
    slack = np.zeros_like(xd)
    slack[..., first:first + n] = 2.0 ** -23 * (r + mate)
    half = 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2
    tol = slack + half * np.abs(want) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    out = got.double().cpu().numpy()
    carried = np.ones(xd.shape[-1], bool)
    carried[first:first + n] = False
    assert np.array_equal(out[..., carried], xd[..., carried])
    assert (np.abs(out - want) <= tol).all(), np.abs(out - want).max()


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("name", list(DTYPES))
@pytest.mark.parametrize("T,H,D,rot,first,inverse", [
    (1, 1, 2, 2, 0, False), (1, 128, 64, 64, 0, False), (3, 5, 7, 4, 1, True),
    (37, 3, 192, 64, 128, False), (130, 64, 128, 64, 0, True), (9, 2, 576, 64, 512, False),
    (2, 3, 1024, 256, 512, True), (2, 1, 1023, 6, 1017, False), (700, 33, 96, 96, 0, False),
    # several heads a thread, vectors of every width, heads left over
    (1000, 7, 130, 98, 0, False), (1200, 8, 132, 100, 32, True), (1100, 5, 125, 90, 3, False),
    (5000, 8, 130, 66, 2, False), (2600, 16, 127, 126, 1, True), (2500, 3, 200, 40, 8, False),
    (90, 9, 1022, 256, 6, False)])
def test_rotation(layout, name, T, H, D, rot, first, inverse):
    import dsa_sparse_indexer_gb300 as dsa
    dtype = DTYPES[name]
    gen = torch.Generator(device="cuda").manual_seed(T + D)
    x = torch.randn((T, H, D), device="cuda", generator=gen).to(dtype)
    cs = RO.table(500, rot, 10000.0).astype(np.float32)
    pos = np.random.default_rng(T).integers(0, 500, T).astype(np.int32)
    g = G.Guards()
    err = dsa.new_error_flags("cuda")
    out = g.empty((T, H, D), dtype)
    got = dsa.rotary_embed(x, G.dev(pos), G.dev(cs), layout, first, inverse, out=out, err_flags=err)
    g.check()
    assert got is out and int(err.item()) == 0
    _check(x, pos, cs, out, layout, first, inverse, dtype)
    # the same in place, and allocated
    held = x.clone()
    assert dsa.rotary_embed(held, G.dev(pos), G.dev(cs), layout, first, inverse, out=held) is held
    assert torch.equal(held, out)
    assert torch.equal(dsa.rotary_embed(x, G.dev(pos), G.dev(cs), layout, first, inverse), out)


@pytest.mark.parametrize("x_at,out_at,width", [(0, 0, 64), (128, 512, 64), (1, 3, 64), (8, 4, 72)])
def test_strided_views(x_at, out_at, width):
    """Part of a wider head in, part of another out; what lies beside the
    output's part stays as it was.  Offsets that leave no 16-byte alignment
    among them."""
    import dsa_sparse_indexer_gb300 as dsa
    T, H, rot = 21, 6, 64
    gen = torch.Generator(device="cuda").manual_seed(5)
    wide = torch.randn((T, H, 200), device="cuda", generator=gen).bfloat16()
    target = torch.full((H, T, 600), 7.0, device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    cs = RO.table(64, rot, 10000.0).astype(np.float32)
    pos = np.arange(T, dtype=np.int32) * 3
    x, out = wide[..., x_at:x_at + width], target[..., out_at:out_at + width]
    before = wide.clone()
    dsa.rotary_embed(x, G.dev(pos), G.dev(cs), "half", out=out)
    torch.cuda.synchronize()
    assert torch.equal(wide, before)
    _check(x, pos, cs, out, "half", 0, False, torch.bfloat16)
    assert (target[..., :out_at] == 7).all() and (target[..., out_at + width:] == 7).all()


def test_two_dimensions_broadcast_input_and_no_tokens():
    import dsa_sparse_indexer_gb300 as dsa
    cs = RO.table(16, 64, 10000.0).astype(np.float32)
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((33, 64), device="cuda", generator=gen).bfloat16()
    pos = np.arange(33, dtype=np.int32) % 16
    got = dsa.rotary_embed(x, G.dev(pos), G.dev(cs))
    _check(x[:, None], pos, cs, got[:, None], "interleaved", 0, False, torch.bfloat16)
    shared = x[:, None].expand(33, 4, 64)            # one key for four heads
    many = dsa.rotary_embed(shared, G.dev(pos), G.dev(cs), out=torch.empty_like(shared.contiguous()))
    assert torch.equal(many, got[:, None].expand(33, 4, 64))
    empty = x[:0]
    assert dsa.rotary_embed(empty, G.dev(pos[:0]), G.dev(cs)).shape == (0, 64)
    with pytest.raises(dsa.DSAError):
        dsa.rotary_embed(shared, G.dev(pos), G.dev(cs), out=shared)
    with pytest.raises(ValueError, match="shape"):
        dsa.rotary_embed(x, G.dev(pos), G.dev(cs), out=got[:, :32])
    with pytest.raises(ValueError, match="per token"):
        dsa.rotary_embed(x, G.dev(pos[:5]), G.dev(cs))
    with pytest.raises(ValueError, match="contiguous"):
        dsa.rotary_embed(x.t(), G.dev(pos), G.dev(cs))


def test_positions_outside_the_table_are_carried_and_flagged():
    import dsa_sparse_indexer_gb300 as dsa
    cs = RO.table(10, 64, 10000.0).astype(np.float32)
    gen = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn((4, 2, 64), device="cuda", generator=gen)
    pos = np.array([10, 3, -1, 2 ** 31 - 1], np.int32)
    err = dsa.new_error_flags("cuda")
    got = dsa.rotary_embed(x, G.dev(pos), G.dev(cs), err_flags=err)
    assert int(err.item()) == dsa.DSA_FLAG_BOUNDS
    _check(x, pos, cs, got, "interleaved", 0, False, torch.float32)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_inverse_is_the_gradient(layout):
    """d/dx of sum(g . rotate(x)) is rotate(g) backwards: against central
    differences of the oracle (a linear map: exact up to fp64 rounding), and
    turning back what was turned."""
    import dsa_sparse_indexer_gb300 as dsa
    rng = np.random.default_rng(8)
    cs = RO.table(30, 8, 100.0).astype(np.float32)
    pos = np.array([5, 29], np.int32)
    x, g = rng.standard_normal((2, 1, 10)), rng.standard_normal((2, 1, 10)).astype(np.float32)
    grad = dsa.rotary_embed(G.dev(g), G.dev(pos), G.dev(cs), layout, first=1, inverse=True)
    want = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = 0.5
        f = lambda v: (g * RO.rotate(v, pos, cs, layout, 1)).sum()      # noqa: E731
        want[i] = f(x + d) - f(x - d)
    np.testing.assert_allclose(grad.cpu().numpy(), want, atol=1e-6)


def test_captured_and_replayed_on_a_side_stream():
    import dsa_sparse_indexer_gb300 as dsa
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn((17, 8, 64), device="cuda", generator=gen).bfloat16()
    pos = G.dev(np.arange(17, dtype=np.int32))
    out = torch.empty_like(x)
    table = torch.empty((32, 64), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            dsa.rope_table(32, 64, out=table)
            dsa.rotary_embed(x, pos, table, out=out)
    table.zero_()
    out.zero_()
    for seed in (1, 2):
        x.copy_(torch.randn(x.shape, device="cuda", generator=gen))
        graph.replay()
        want = dsa.rotary_embed(x, pos, dsa.rope_table(32, 64))
        assert torch.equal(out, want)
