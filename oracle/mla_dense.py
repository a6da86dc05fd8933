"""Latent attention over whole contexts, in fp64: the expanded form over a
ragged batch and the absorbed form over each shard's paged cache.  Test
infrastructure.

Both are the softmax definition, written out: s_j = scale * (q . k_j) over the
keys a query sees, O = sum_j exp(s_j) v_j / sum_j exp(s_j), lse2 = log2 sum_j
exp(s_j); a query that sees nothing has O = 0 and lse2 = -inf.  Beside them come
what the tests' bounds need: size = sum_j exp(s_j) |v_j| / sum_j exp(s_j), and
reach = the largest scale * sum_d |q_d k_jd| over the seen keys.
"""
from __future__ import annotations

import numpy as np

from . import dcp_layout as L

LN2 = np.log(2.0)


def attend(q, k, v, scale: float, seen):
    """q [rows, d], k [keys, d], v [keys, e] fp64; seen [rows, keys] bool.
    Returns (out [rows, e], lse2 [rows], size [rows, e], reach [rows])."""
    rows, e = q.shape[0], v.shape[1]
    out, size = np.zeros((rows, e)), np.zeros((rows, e))
    lse2, reach = np.full(rows, -np.inf), np.zeros(rows)
    for i in range(rows):
        js = np.nonzero(seen[i])[0]
        if js.size == 0:
            continue
        s = scale * (k[js] @ q[i])
        m = s.max()
        w = np.exp(s - m)
        out[i] = w @ v[js] / w.sum()
        size[i] = w @ np.abs(v[js]) / w.sum()
        lse2[i] = (m + np.log(w.sum())) / LN2
        reach[i] = abs(scale) * (np.abs(k[js]) @ np.abs(q[i])).max()
    return out, lse2, size, reach


def prefill(q, k_nope, k_pe, v, cu_q, cu_k, scale: float, causal: bool):
    """q [Tq, H, 192], k_nope [Tk, H, 128], k_pe [Tk, 64], v [Tk, H, 128] fp64.
    Rows of no sequence are NaN in every result."""
    Tq, H, _ = q.shape
    out, size = np.full((Tq, H, v.shape[2]), np.nan), np.full((Tq, H, v.shape[2]), np.nan)
    lse2, reach = np.full((Tq, H), np.nan), np.full((Tq, H), np.nan)
    for i in range(len(cu_q) - 1):
        qs, ks = slice(cu_q[i], cu_q[i + 1]), slice(cu_k[i], cu_k[i + 1])
        lq, lk = cu_q[i + 1] - cu_q[i], cu_k[i + 1] - cu_k[i]
        seen = np.ones((lq, lk), bool)
        if causal:
            seen = np.arange(lk)[None] <= np.arange(lq)[:, None] + (lk - lq)
        for h in range(H):
            k = np.concatenate([k_nope[ks, h], k_pe[ks]], axis=1)
            out[qs, h], lse2[qs, h], size[qs, h], reach[qs, h] = attend(q[qs, h], k, v[ks, h], scale, seen)
    return out, lse2, size, reach


def decode(q, cache, table, block_size: int, starts, lens, S: int, I: int, scale: float,
           tree_mask=None, d_v: int = 512):
    """q [rows, H, 576], cache [S, n_slots, 576] fp64, table [S, reqs, cols]
    int32, tree_mask [rows, words] int32 or None.  Results [S, rows, H, ...]; rows
    of no request are NaN; a token whose table entry lies outside the cache is
    left out."""
    rows, H, _ = q.shape
    out, size = np.full((S, rows, H, d_v), np.nan), np.full((S, rows, H, d_v), np.nan)
    lse2, reach = np.full((S, rows, H), np.nan), np.full((S, rows, H), np.nan)
    for r, length in enumerate(lens):
        n = starts[r + 1] - starts[r]
        for s in range(S):
            tokens = np.asarray(L.owned_tokens(max(int(length), 0), s, S, I), np.int64)
            local = np.arange(tokens.size)
            there = local < table.shape[2] * block_size
            tokens, local = tokens[there], local[there]
            entry = table[s, r, local // block_size].astype(np.int64)
            slot = entry * block_size + local % block_size
            there = (entry >= 0) & (slot < cache.shape[1])
            tokens, k = tokens[there], cache[s, slot[there]]
            for j in range(n):
                row = starts[r] + j
                i = tokens - (int(length) - n)
                if tree_mask is None:
                    see = i <= j
                else:
                    word = np.clip(i, 0, None) // 32
                    inside = word < tree_mask.shape[1]
                    bits = tree_mask[row, np.minimum(word, tree_mask.shape[1] - 1)].astype(np.int64)
                    see = (i < 0) | (inside & ((bits >> (np.clip(i, 0, None) % 32)) & 1 == 1))
                o, l2, sz, rc = attend(q[row], k, k[:, :d_v], scale, np.tile(see, (H, 1)))
                out[s, row], lse2[s, row], size[s, row], reach[s, row] = o, l2, sz, rc
    return out, lse2, size, reach
