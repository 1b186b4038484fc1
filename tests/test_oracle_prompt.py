"""The prompt path's oracles pinned: chunk and windowed attention against the tree oracle, dense softmax and closed
forms, log probabilities against scipy."""
import math

import numpy as np
import pytest
import scipy.special

import oracle
import workloads as W


def _chunk_inputs(lens, prefix, Hq, Hkv, D, bs, seed=0):
    kv = [p + n for p, n in zip(prefix, lens)]
    table, nblk = W.paged_layout(W.rng(seed, "table"), np.array(kv, np.int32), bs, True)
    cu = np.concatenate(([0], np.cumsum(lens)))
    q = W.normal_bf16(seed, "q", (int(cu[-1]), Hq, D))
    k, v = (W.normal_bf16(seed, n, (nblk, Hkv, bs, D)) for n in ("k", "v"))
    return q, k, v, table, cu, np.array(kv)


def test_chunk_of_a_whole_prompt_is_dense_causal_softmax():
    q, k, v, table, cu, kv = _chunk_inputs([9, 4], [0, 3], 4, 2, 64, 16)
    out, lse = oracle.window.chunk_attention(q, k, v, table, cu, kv)
    f = oracle.attention.bf16_to_f64
    for b in range(2):
        n, T = cu[b + 1] - cu[b], kv[b]
        for h in range(4):
            keys = oracle.attention.prefix_kv(k, table, b, h // 2, T, 16)
            vals = oracle.attention.prefix_kv(v, table, b, h // 2, T, 16)
            s = f(q[cu[b]:cu[b + 1], h]) @ keys.T / 8.0
            s[np.triu_indices(n, T - n + 1, T)] = -np.inf
            np.testing.assert_allclose(out[cu[b]:cu[b + 1], h], scipy.special.softmax(s, axis=1) @ vals, atol=1e-12)
            np.testing.assert_allclose(lse[cu[b]:cu[b + 1], h], scipy.special.logsumexp(s, axis=1), atol=1e-12)


def test_a_chunk_is_a_chain_tree_whose_keys_are_cached():
    """The chunk's rows with the keys before it as prefix and its own as a chain tree."""
    q, k, v, table, cu, kv = _chunk_inputs([7], [21], 2, 1, 64, 16, seed=3)
    out, lse = oracle.window.chunk_attention(q, k, v, table, cu, kv)
    own = [(c[table[0, t // 16], :, t % 16])[None] for c in (k, v) for t in range(21, 28)]
    kt, vt = np.concatenate(own[:7])[None], np.concatenate(own[7:])[None]
    chain = W.tree_chain(7)[None]
    o2, l2 = oracle.attention.tree_attention(q[None], k, v, table, np.array([21]), kt, vt, chain)
    np.testing.assert_allclose(out, o2[0], atol=1e-12)
    np.testing.assert_allclose(lse, l2[0], atol=1e-12)


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 0), (5, 3), (1, 40), (100, 2)])
def test_windows_by_enumeration(window, sinks):
    for p in range(30):
        for t in range(30):
            want = t in set(range(max(0, p - window + 1), p + 1)) | set(range(min(sinks, p + 1)))
            assert bool(oracle.window.near(np.array(p), np.array(t), window, sinks)) == want


def test_a_window_of_one_without_sinks_copies_the_value():
    q, k, v, table, cu, kv = _chunk_inputs([5], [6], 2, 1, 64, 16, seed=5)
    out, _ = oracle.window.chunk_attention(q, k, v, table, cu, kv, window=1)
    for i in range(5):
        t = 6 + i
        np.testing.assert_array_equal(out[i, 0], oracle.attention.bf16_to_f64(v[table[0, t // 16], 0, t % 16]))


def test_a_window_past_everything_is_the_tree_oracle():
    g = W.rng(2, "t")
    parent = np.stack([W.tree_random_levels(g, 12, 4) for _ in range(2)])
    c = W.build_case("w", 2, parent, [19, 0], 4, 2, 64, 16, True)
    a = (c.q, c.k_cache, c.v_cache, c.block_table, c.prefix_len, c.k_tree, c.v_tree, c.parent)
    out, lse = oracle.attention.tree_attention(*a)
    o2, l2 = oracle.window.tree_attention(*a, window=1000, sinks=0)
    np.testing.assert_allclose(o2, out, atol=1e-12)
    np.testing.assert_allclose(l2, lse, atol=1e-12)
    o3, _ = oracle.window.tree_attention(*a, window=1, sinks=1000)  # sinks past everything too
    np.testing.assert_allclose(o3, out, atol=1e-12)


def test_a_windowed_chain_tree_is_a_windowed_chunk():
    q, k, v, table, cu, kv = _chunk_inputs([9], [30], 2, 2, 64, 16, seed=8)
    out, lse = oracle.window.chunk_attention(q, k, v, table, cu, kv, window=4, sinks=2)
    own = [(c[table[0, t // 16], :, t % 16])[None] for c in (k, v) for t in range(30, 39)]
    o2, l2 = oracle.window.tree_attention(q[None], k, v, table, np.array([30]), np.concatenate(own[:9])[None],
                                          np.concatenate(own[9:])[None], W.tree_chain(9)[None], 4, 2)
    np.testing.assert_allclose(out, o2[0], atol=1e-12)
    np.testing.assert_allclose(lse, l2[0], atol=1e-12)


def test_logprobs_against_scipy():
    x = W.rng(1, "x").standard_normal((4, 50)).astype(np.float32) * 3
    x[1, 7:20] = -np.inf
    t = [3, 2, 49, 0]
    for temp in (1.0, 0.5):
        lp, ent, ids, alt = oracle.logprobs.score(x, t, temperature=temp, top=3)
        ref = scipy.special.log_softmax(x.astype(np.float64) / temp, axis=1)
        np.testing.assert_allclose(lp, ref[np.arange(4), t], atol=1e-12)
        np.testing.assert_allclose(ent, scipy.special.entr(np.exp(ref)).sum(axis=1), atol=1e-12)
        np.testing.assert_array_equal(ids, np.argsort(-x, axis=1, kind="stable")[:, :3])
        np.testing.assert_allclose(alt, np.take_along_axis(ref, ids, axis=1), atol=1e-12)


def test_logprobs_closed_forms():
    x = np.full((5, 8), -np.inf)
    x[0] = 2.5                      # uniform: ln 8, ties by index
    x[1, 5] = 1.0                   # one token
    x[3, [2, 6]] = [0.0, math.log(3)]  # 1/4, 3/4
    x[4] = np.finfo(np.float32).min    # the type's lowest value everywhere: uniform
    lp, ent, ids, alt = oracle.logprobs.score(x, [4, 5, 0, 2, -1], top=3)
    np.testing.assert_allclose(lp, [-math.log(8), 0, -np.inf, -math.log(4), 0], atol=1e-15)
    h = -0.25 * math.log(0.25) - 0.75 * math.log(0.75)
    np.testing.assert_allclose(ent, [math.log(8), 0, 0, h, math.log(8)], atol=1e-15)
    assert ids.tolist() == [[0, 1, 2], [5, -1, -1], [-1] * 3, [6, 2, -1], [0, 1, 2]]
    assert alt[2].tolist() == [-np.inf] * 3
    lp, _, ids, _ = oracle.logprobs.score(x, [9, 1], rows=[0, 7], top=1)
    assert np.isnan(lp).all() and ids.tolist() == [[0], [-2]]
