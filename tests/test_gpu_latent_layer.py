"""The operators together, as a layer uses them: a prompt prefilled with expanded
heads while its cache rows and indexer keys are written; drafted tokens verified by
the absorbed attention over that cache, which must give the same outputs; the
indexer over its own keys, whose selection of every token must give them too."""
import numpy as np
import pytest
import torch

from oracle import mla_dense as MD

pytestmark = pytest.mark.gpu

H, DN, DR, DV, DL = 16, 128, 64, 128, 512
S, I, BLOCK = 2, 4, 64
SCALE = 192.0 ** -0.5


def layer(T, n, seed=0):
    """A sequence of T tokens whose last n are drafts, through both forms."""
    import dsa_sparse_indexer_gb300 as dsa
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, device="cuda", generator=g)   # noqa: E731
    cs = dsa.rope_table(4096, DR)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    w_uk, w_uv = r(H, DN, DL) / DL ** 0.5, r(H, DL, DV) / DL ** 0.5
    q_nope = r(T, H, DN).bfloat16()
    q_pe = dsa.rotary_embed(r(T, H, DR).bfloat16(), pos, cs)
    kv, kpe = dsa.fused_norm_rope(r(T, DL).bfloat16(), r(T, DR).bfloat16(), pos, torch.ones(DL, device="cuda"), 1e-6, cs)
    # the cache: every shard's slots of the tokens
    cols = -(-(T // S + I) // BLOCK)
    table = torch.stack([torch.randperm(cols + 2, device="cuda", generator=g)[:cols] for _ in range(S)]).int().view(S, 1, cols)
    slots = dsa.slot_mapping(pos, table, BLOCK, I, token_req=torch.zeros_like(pos))
    cache = torch.zeros((S, (cols + 2) * BLOCK, DL + DR), dtype=torch.bfloat16, device="cuda")
    for s in range(S):
        dsa.kv_cache_insert(kv, kpe, slots[s].contiguous(), cache[s])
    return dict(cs=cs, pos=pos, w_uk=w_uk, w_uv=w_uv, q_nope=q_nope, q_pe=q_pe, kv=kv, kpe=kpe, table=table,
                cache=cache, slots=slots, g=g)


@pytest.mark.parametrize("T,n,tree", [(300, 1, False), (517, 8, False), (700, 40, True)])
def test_expanded_and_absorbed_agree(T, n, tree):
    import dsa_sparse_indexer_gb300 as dsa
    L = layer(T, n, seed=T)
    # absorbed: each head's query through W_uk, outputs through W_uv
    q_lat = torch.einsum("thd,hdl->thl", L["q_nope"][-n:].float(), L["w_uk"])
    q = torch.cat([q_lat, L["q_pe"][-n:].float()], -1).bfloat16()
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    mask = None
    if tree:                                      # every draft sees itself and two steps back
        bits = torch.zeros((n, 64), dtype=torch.long)
        for j in range(n):
            for i in (j, j - 3, j - 9):
                if i >= 0:
                    bits[j, i] = 1
        w = (bits.view(n, 2, 32) << torch.arange(32)).sum(-1)
        mask = torch.where(w >= 1 << 31, w - (1 << 32), w).int().cuda()
    part, lse2 = dsa.mla_decode(q, L["cache"], L["table"], BLOCK, starts, lens, I, SCALE, tree_mask=mask)
    o, lse = dsa.lse_combine(part, lse2)
    absorbed = torch.einsum("thl,hlv->thv", o.float(), L["w_uv"])
    # expanded: the latents through both, rows of the drafts alone
    k = torch.einsum("tl,hdl->thd", L["kv"].float(), L["w_uk"]).bfloat16()
    v = torch.einsum("tl,hlv->thv", L["kv"].float(), L["w_uv"]).bfloat16()
    qe = torch.cat([L["q_nope"][-n:], L["q_pe"][-n:]], -1)
    if not tree:
        cu_k = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        out, lse2e = dsa.mla_prefill(qe, k, L["kpe"], v, starts, cu_k, SCALE)
        expanded = out.float()
        assert (lse / np.log(2.0) - lse2e).abs().max() <= 0.15
    else:
        seen = torch.ones((n, T), dtype=torch.bool, device="cuda")
        seen[:, T - n:] = bits[:, :n].bool().cuda()
        f = lambda t: t.double().cpu().numpy()   # noqa: E731
        expanded = torch.stack([torch.from_numpy(MD.attend(
            f(qe[:, h]), np.concatenate([f(k[:, h]), f(L["kpe"])], 1), f(v[:, h]), SCALE, seen.cpu().numpy())[0])
            for h in range(H)], 1).float().cuda()
    err = (absorbed - expanded).abs()
    assert err.max() <= 0.06 * v.float().abs().max() and err.mean() <= 0.01 * v.float().abs().mean()


def test_indexer_selects_over_its_cache():
    """Keys inserted and queries made here, logits, local top-K, merge, conversion:
    with more places than tokens every token is selected, and the sparse attention
    over the selection is the dense one."""
    import dsa_sparse_indexer_gb300 as dsa
    T, n, K = 400, 3, 512
    L = layer(T, n, seed=7)
    r = lambda *s: torch.randn(s, device="cuda", generator=L["g"])   # noqa: E731
    keys = torch.zeros((S, L["cache"].shape[1], 128), dtype=torch.uint8, device="cuda")
    dsa.indexer_key_insert(r(T, 128).bfloat16(), torch.ones(128, device="cuda"), None, 1e-6, L["pos"], L["cs"],
                           L["slots"], keys)
    at = L["pos"][-n:].contiguous()
    q8, w8 = dsa.indexer_query_fp8(r(n, 64, 128).bfloat16(), r(n, 64), at, L["cs"], factor=128.0 ** -0.5 / 8)
    ends, req, ld = at + 1, torch.zeros_like(at), 8192
    logits = dsa.indexer_logits(q8, w8, keys, L["table"], BLOCK, ends, I, ld, row_to_req=req)
    assert torch.isfinite(logits[:, :, :100]).all()
    _, cand = dsa.shard_topk_pack(logits, ends, K, I)
    ids = dsa.merge_topk_stable(cand, K)
    assert all(sorted(x for x in row.tolist() if x >= 0) == list(range(int(e))) for row, e in zip(ids, ends))
    slots, counts = dsa.convert_index_compact(ids, L["table"], BLOCK, I, row_to_req=req)
    q = torch.randn((n, 64, 576), device="cuda", generator=L["g"]).bfloat16()
    sparse, l2 = dsa.sparse_mla_decode(q, L["cache"], slots, counts, SCALE)
    dense, d2 = dsa.mla_decode(q, L["cache"], L["table"], BLOCK, torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                               torch.tensor([T], dtype=torch.int32, device="cuda"), I, SCALE)
    assert (l2 - d2).abs().max() <= 2e-3
    assert (sparse.float() - dense.float()).abs().max() <= 4 * 2.0 ** -8 * L["cache"].float().abs().max()


def test_inference_mode_and_versions():
    """Outputs that the caller gave count as changed; tensors made under
    inference_mode, which have no version, are taken as well."""
    import dsa_sparse_indexer_gb300 as dsa
    T, heads = 3, 2

    def run(given):
        q, kv = torch.zeros(T, heads, 192, device="cuda").half(), torch.zeros(T, heads, 256, device="cuda").half()
        cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        o, l2 = torch.ones(T, heads, 128, device="cuda").half(), torch.ones(T, heads, device="cuda")
        dsa.mla_prefill(q, kv[..., :128], torch.zeros(T, 64, device="cuda").half(), kv[..., 128:], cu, cu, 1.0,
                        out=o if given else None, lse2=l2 if given else None)
        cache = torch.zeros(1, 64, 576, device="cuda").bfloat16()
        o2 = torch.ones(1, T, heads, 512, device="cuda").bfloat16()
        dsa.mla_decode(torch.zeros(T, heads, 576, device="cuda").bfloat16(), cache,
                       torch.zeros(1, 1, 1, dtype=torch.int32, device="cuda"), 64, cu,
                       torch.tensor([T], dtype=torch.int32, device="cuda"), 1, 1.0, out=o2 if given else None)
        cs, pos = dsa.rope_table(8, 64), torch.arange(T, dtype=torch.int32, device="cuda")
        keys = torch.zeros(1, 64, 128, dtype=torch.uint8, device="cuda")
        dsa.indexer_key_insert(torch.zeros(T, 128, device="cuda").bfloat16(), torch.ones(128, device="cuda"), None, 1e-6,
                               pos, cs, pos.view(1, T), keys)
        w = torch.ones(T, heads, device="cuda")
        dsa.indexer_query_fp8(torch.zeros(T, heads, 128, device="cuda").bfloat16(), w, pos, cs,
                              weights_out=w if given else None)
        torch.cuda.synchronize()
        return o, l2, o2, keys, w

    for given in (False, True):
        with torch.inference_mode():
            run(given)
    before = [t._version for t in run(False)]
    after = [t._version for t in run(True)]
    assert [b - a for a, b in zip(before, after)] == [1, 1, 1, 0, 1] and before[3] > 0
