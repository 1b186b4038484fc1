"""Oracle: attention of a chunk of cached tokens, and of a tree in a windowed layer (test infrastructure only).

By definition, a row and a key at a time, in fp64.  A row at position p sees a key at position t iff t <= p and it is
near: no window, or p - t < window, or t < sinks (P2 How It Works: a token attends to what is before it and itself).

chunk_attention: sequence b has kv_len[b] tokens in the paged cache, the last cu_len[b+1] - cu_len[b] of which are the
rows.  tree_attention: the rows are tree nodes at prefix_len + depth; among the nodes only ancestors and the node itself
are keys.  A row that sees nothing gives zeros and an lse of -inf.
"""
from __future__ import annotations

import numpy as np

from .attention import bf16_to_f64, prefix_kv
from .tree import ancestry_matrix


def near(p, t, window, sinks):
    """Whether position p is within reach of position t (both numpy, broadcast)."""
    if window == 0:
        return t <= p
    return (t <= p) & ((p - t < window) | (t < sinks))


def attend(q, keys, vals, visible, scale):
    """q [R, D], keys, vals [T, D], visible [R, T] -> out [R, D], lse [R]; only visible keys enter a row's sums."""
    out = np.zeros(q.shape)
    lse = np.full(q.shape[0], -np.inf)
    for r in range(q.shape[0]):
        at = np.flatnonzero(visible[r])
        if not len(at):
            continue
        s = scale * (keys[at] @ q[r])
        m = s.max()
        w = np.exp(s - m)
        out[r] = w @ vals[at] / w.sum()
        lse[r] = m + np.log(w.sum())
    return out, lse


def chunk_attention(q, k_cache, v_cache, block_table, cu_len, kv_len, scale=0.0, window=0, sinks=0):
    """q [T, Hq, D], caches [blocks, Hkv, bs, D]: bf16 bits -> out [T, Hq, D], lse [T, Hq]; rows of no sequence NaN."""
    T, Hq, D = q.shape
    Hkv, bs = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hkv
    scale = scale or 1.0 / np.sqrt(D)
    out, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    for b in range(len(kv_len)):
        lo, hi, kv = int(cu_len[b]), int(cu_len[b + 1]), int(kv_len[b])
        if hi == lo:
            continue
        pos = np.arange(kv - (hi - lo), kv)
        vis = near(pos[:, None], np.arange(kv)[None], window, sinks)
        seen = np.flatnonzero(vis.any(axis=0))  # keys that no row sees are never looked up
        for g in range(Hkv):
            keys, vals = (np.zeros((kv, D)) for _ in range(2))
            for t in seen:
                blk = int(block_table[b, t // bs])
                keys[t], vals[t] = bf16_to_f64(k_cache[blk, g, t % bs]), bf16_to_f64(v_cache[blk, g, t % bs])
            for h in range(g * G, (g + 1) * G):
                out[lo:hi, h], lse[lo:hi, h] = attend(bf16_to_f64(q[lo:hi, h]), keys, vals, vis, scale)
    return out, lse


def tree_attention(q, k_cache, v_cache, block_table, prefix_len, k_tree, v_tree, parent, window, sinks, scale=0.0):
    """The same of a tree's nodes: q [B, N, Hq, D], parent [B, N] -> out [B, N, Hq, D], lse [B, N, Hq]."""
    B, N, Hq, D = q.shape
    Hkv, bs = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hkv
    scale = scale or 1.0 / np.sqrt(D)
    out, lse = np.zeros((B, N, Hq, D)), np.zeros((B, N, Hq))
    for b in range(B):
        P = int(prefix_len[b])
        depth = np.zeros(N, np.int64)
        for i in range(N):
            if parent[b, i] >= 0:
                depth[i] = depth[parent[b, i]] + 1
        pos = P + depth
        own = ancestry_matrix(parent[b]) & near(pos[:, None], pos[None], window, sinks)
        vis = np.concatenate([near(pos[:, None], np.arange(P)[None], window, sinks), own], axis=1)
        for g in range(Hkv):
            keys = np.concatenate([prefix_kv(k_cache, block_table, b, g, P, bs), bf16_to_f64(k_tree[b, :, g])])
            vals = np.concatenate([prefix_kv(v_cache, block_table, b, g, P, bs), bf16_to_f64(v_tree[b, :, g])])
            for h in range(g * G, (g + 1) * G):
                out[b, :, h], lse[b, :, h] = attend(bf16_to_f64(q[b, :, h]), keys, vals, vis, scale)
    return out, lse
