"""tree_attn_fwd_window against the fp64 oracle, over pools that hold NaN wherever no node may look."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from tests.gpu_util import to_dev
from tests.prompt_util import NAN, assert_rows, f64, live_keys

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_attention_speculative_gb300 import _build
    _build.build()


def build(N, kind, prefix, Hq, Hkv, D, bs, window, sinks, seed=0):
    g = W.rng(seed, "tree")
    make = {"chain": lambda: W.tree_chain(N), "star": lambda: W.tree_star(N),
            "random": lambda: W.tree_random_recursive(g, N)}[kind]
    c = W.build_case("win", seed, np.stack([make() for _ in prefix]), prefix, Hq, Hkv, D, bs, True)
    k, v, table = np.full_like(c.k_cache, NAN), np.full_like(c.v_cache, NAN), np.full_like(c.block_table, 1 << 20)
    for b, P in enumerate(prefix):
        t = live_keys(P, 1, window, sinks)  # those that the root sees
        t = t[t < P]
        blk = c.block_table[b, t // bs]
        table[b, t // bs] = blk
        k[blk, :, t % bs], v[blk, :, t % bs] = c.k_cache[blk, :, t % bs], c.v_cache[blk, :, t % bs]
    args = (c.q, np.where(k == NAN, 0, k), np.where(v == NAN, 0, v), c.block_table, c.prefix_len, c.k_tree)
    ref = oracle.window.tree_attention(*args, c.v_tree, c.parent, window, sinks)
    mag, _ = oracle.window.tree_attention(args[0], args[1], args[2] & 0x7FFF, *args[3:], c.v_tree & 0x7FFF, c.parent, window,
                                          sinks)
    c.k_cache, c.v_cache, c.block_table = k, v, table
    return c, (*ref, mag)


def run(c, window, sinks, forest=False):
    from tree_attention_speculative_gb300.step import TreeVerifyStep
    t = to_dev(c)
    step = TreeVerifyStep(c.B, c.N, c.Hq, c.Hkv, c.D, c.prefix_len, window=window, sinks=sinks, forest=forest)
    step.run(t["parent"], t["prefix_len"], t["q"], t["k_cache"], t["v_cache"], t["block_table"], t["k_tree"], t["v_tree"])
    torch.cuda.synchronize()
    assert (step.ws_attn[:256] == 0).all()
    return step


CASES = [
    # N, tree, prefix, Hq, Hkv, D, bs, window, sinks
    (1, "chain", [0, 300], 8, 2, 128, 16, 64, 4),
    (5, "random", [16], 2, 2, 64, 16, 8, 2),
    (26, "random", [0, 1000, 129, 5], 8, 2, 128, 16, 100, 4),
    (40, "chain", [257, 3], 16, 1, 64, 128, 7, 0),        # a chain longer than the window: ancestors fall out
    (40, "chain", [1, 30], 4, 2, 128, 48, 5, 9),           # and some of them are sinks
    (130, "chain", [500], 2, 1, 128, 16, 70, 3),           # three mask words
    (256, "chain", [40], 1, 1, 64, 32, 200, 50),           # four, two tree tiles
    (200, "random", [700, 90], 4, 4, 128, 16, 1, 0),       # a node sees itself alone
    (64, "star", [2000], 8, 1, 128, 144, 256, 130),
    (9, "random", [6000, 6000], 8, 8, 128, 64, 4096, 4),   # a long window, cut
    (37, "random", [300, 0], 8, 2, 64, 80, 1 << 30, 0),    # a window past everything
    (12, "chain", [50], 4, 2, 128, 16, 3, 1 << 30),        # sinks past everything
]


@pytest.mark.parametrize("N,kind,prefix,Hq,Hkv,D,bs,window,sinks", CASES)
def test_matches_oracle(N, kind, prefix, Hq, Hkv, D, bs, window, sinks):
    c, ref = build(N, kind, prefix, Hq, Hkv, D, bs, window, sinks, seed=N + D)
    step = run(c, window, sinks)
    assert step.status.cpu().tolist() == [0] * c.B
    assert_rows(f64(step.out), f64(step.lse), *ref)


def test_a_window_past_everything_agrees_with_tree_attn_fwd():
    from tree_attention_speculative_gb300.step import TreeVerifyStep
    c = W.build_case("w", 5, np.stack([W.tree_random_recursive(W.rng(5, "t"), 50)] * 3), [700, 64, 0], 8, 2, 128, 16, True)
    t = to_dev(c)
    outs = []
    for window in (0, 1 << 20):
        step = TreeVerifyStep(c.B, c.N, c.Hq, c.Hkv, c.D, c.prefix_len, window=window)
        step.run(t["parent"], t["prefix_len"], t["q"], t["k_cache"], t["v_cache"], t["block_table"], t["k_tree"], t["v_tree"])
        outs.append((f64(step.out), f64(step.lse)))
    np.testing.assert_allclose(outs[0][0], outs[1][0], atol=2.0 ** -6, rtol=2.0 ** -6)
    np.testing.assert_allclose(outs[0][1], outs[1][1], atol=2.0 ** -10)


def test_rows_that_see_nothing_give_zeros():
    import tree_attention_speculative_gb300 as ts
    from tree_attention_speculative_gb300.step import TreeVerifyStep
    c = W.build_case("w", 6, np.stack([W.tree_chain(6)] * 2), [0, 40], 4, 2, 128, 16, True)
    t = to_dev(c)
    step = TreeVerifyStep(c.B, c.N, c.Hq, c.Hkv, c.D, c.prefix_len, window=4)
    step.ancestry(t["parent"], t["prefix_len"])
    step.anc[0, 3] = 0  # no prefix, an empty mask row
    # the key of a node hidden from every row may hold anything
    step.anc[:, :, 0] &= ~(1 << 5)
    t["k_tree"][:, 5] = float("nan")
    step.attention(t["q"], t["k_cache"], t["v_cache"], t["block_table"], t["prefix_len"], t["k_tree"], t["v_tree"])
    torch.cuda.synchronize()
    assert (f64(step.out)[0, 3] == 0).all() and np.isneginf(f64(step.lse)[0, 3]).all()
    assert np.isfinite(f64(step.out)).all()
    assert ts.STATUS[step.status.cpu().tolist()[0]] == "TS_OK"


def test_forests_and_a_bad_prefix():
    parent = np.array([[-1, 0, -1, 2, 3, -1]] * 2, np.int32)
    c = W.build_case("w", 7, parent, [100, 90], 4, 2, 64, 16, True)
    step = run(c, 50, 2, forest=True)
    # each root's tree by itself: the oracle on the trees, whose nodes keep their order
    for nodes in ([0, 1], [2, 3, 4], [5]):
        sub = np.array([[-1] + list(range(len(nodes) - 1))] * 2, np.int32)
        args = (c.q[:, nodes], c.k_cache, c.v_cache, c.block_table, c.prefix_len, c.k_tree[:, nodes])
        out, lse = oracle.window.tree_attention(*args, c.v_tree[:, nodes], sub, 50, 2)
        mag, _ = oracle.window.tree_attention(args[0], args[1], args[2] & 0x7FFF, *args[3:], c.v_tree[:, nodes] & 0x7FFF, sub, 50, 2)
        assert_rows(f64(step.out)[:, nodes], f64(step.lse)[:, nodes], out, lse, mag)
    t = to_dev(c)
    step.out.fill_(7.0)
    t["prefix_len"][1] = 1 << 29
    step.attention(t["q"], t["k_cache"], t["v_cache"], t["block_table"], t["prefix_len"], t["k_tree"], t["v_tree"])
    torch.cuda.synchronize()
    assert step.status.cpu().tolist() == [0, -2]
    assert (f64(step.out)[1] == 7).all()


def test_an_empty_mask_row_is_a_node_at_depth_0():
    """It sees what the root sees of the prefix, and no node; the pool is NaN at what the root does not see."""
    window, sinks, P = 20, 3, 300
    c, _ = build(6, "chain", [P, 7], 4, 2, 128, 16, window, sinks, seed=9)
    t = to_dev(c)
    from tree_attention_speculative_gb300.step import TreeVerifyStep
    step = TreeVerifyStep(c.B, c.N, c.Hq, c.Hkv, c.D, c.prefix_len, window=window, sinks=sinks)
    step.ancestry(t["parent"], t["prefix_len"])
    step.anc[:, 2] = 0
    step.attention(t["q"], t["k_cache"], t["v_cache"], t["block_table"], t["prefix_len"], t["k_tree"], t["v_tree"])
    torch.cuda.synchronize()
    at = live_keys(P, 1, window, sinks)
    at = at[at < P]
    bits = oracle.attention.bf16_to_f64
    for h in range(c.Hq):
        keys, vals = (bits(x[c.block_table[0, at // 16], h // 2, at % 16]) for x in (c.k_cache, c.v_cache))
        seen = np.ones((1, len(at)), bool)
        out, lse = oracle.window.attend(bits(c.q[0, 2, h])[None], keys, vals, seen, 128 ** -0.5)
        mag, _ = oracle.window.attend(bits(c.q[0, 2, h])[None], keys, np.abs(vals), seen, 128 ** -0.5)
        assert_rows(f64(step.out)[0, 2, h][None], f64(step.lse)[0, 2, h][None], out, lse, mag)
    assert np.isfinite(f64(step.out)).all()


def test_a_captured_call_follows_the_prefix():
    import tree_attention_speculative_gb300 as ts
    window, sinks = 40, 5
    start, end = [200, 0, 30], [391, 64, 1000]
    c, _ = build(9, "random", end, 4, 1, 128, 16, 1 << 20, 0, seed=11)  # (all of the pool is there)
    t = to_dev(c)
    out = torch.zeros((c.B, c.N, c.Hq, c.D), dtype=torch.bfloat16, device="cuda")
    lse, status = torch.zeros((c.B, c.N, c.Hq), device="cuda"), torch.zeros(c.B, dtype=torch.int32, device="cuda")
    from tree_attention_speculative_gb300.step import TreeVerifyStep
    step = TreeVerifyStep(c.B, c.N, c.Hq, c.Hkv, c.D, end, window=window, sinks=sinks)
    step.ancestry(t["parent"], t["prefix_len"])
    p = ts.attn_params(t["q"], t["k_cache"], t["v_cache"], t["block_table"], t["prefix_len"], np.array(start, np.int32),
                       t["k_tree"], t["v_tree"], step.anc, None, out, lse, status)
    ws = torch.zeros(ts.tree_attn_window_workspace_size(p, window, sinks), dtype=torch.uint8, device="cuda")
    ts.tree_attn_fwd_window(p, window, sinks, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ts.tree_attn_fwd_window(p, window, sinks, ws)
    for P in (start, end):
        t["prefix_len"].copy_(torch.tensor(P, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        a = (c.q, c.k_cache, c.v_cache, c.block_table, np.array(P, np.int32), c.k_tree)
        ref = oracle.window.tree_attention(*a, c.v_tree, c.parent, window, sinks)
        mag, _ = oracle.window.tree_attention(a[0], a[1], a[2] & 0x7FFF, *a[3:], c.v_tree & 0x7FFF, c.parent, window, sinks)
        assert status.cpu().tolist() == [0] * 3
        assert_rows(f64(out), f64(lse), *ref, mag)


def test_more_sequences_than_a_launch_takes():
    prefix = [(b * 53) % 150 for b in range(260)]
    c, ref = build(3, "random", prefix, 2, 1, 64, 16, 12, 2, seed=13)
    step = run(c, 12, 2)
    assert step.status.cpu().tolist() == [0] * c.B
    assert_rows(f64(step.out), f64(step.lse), *ref)
