"""Chunk and windowed attention where one key outweighs all the others: its weight's rounding to bf16 cancels against the
sum that the output is divided by, so that the output is that key's value to the bit.

Logits are exact (channels of q are all c, those of a key all w, scale 1 / D: a logit of c w).  The first keys, and so every
reference, have a logit of 0, one key of a later tile one of 17 to 23, so its weight is anywhere between two bf16 numbers.
The others together have 3000 e^-17 < 2^-12.9 of it, and values within 2^-4, so they move the output by less than 2^-16;
what the hot key's value (mantissa 255/128: steps of 2^-7) lacks to itself is then fp32's.  An error of 2^-8 of the weight would
be as much of the value, up to twice what rounding to it lets pass.

lse: the sum of the weights before rounding, in fp32, within 2^-17 of a logit of up to 23 (exp2 and log2 to 2^-21 of
themselves, a few steps of 2^-19)."""
import numpy as np
import pytest
import torch

import workloads as W
from tests.gpu_util import to_dev
from tests.prompt_util import Chunk, f64

pytestmark = pytest.mark.gpu

HOT = 255 / 128  # the hot key's value, 0x3FFF


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_attention_speculative_gb300 import _build
    _build.build()


def bits(x):
    return (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def cold(shape, seed):
    """Values within 2^-4."""
    return bits(np.random.default_rng(seed).choice(np.float32([-1, -0.5, 0.5, 1]), shape) / 16)


def check(out, lse, factor, n_others):
    """factor: each row's c; the hot key's w is 16."""
    assert (out == HOT).all(), (int((out != HOT).sum()), out.size)
    want = 16 * factor + np.log1p(n_others * np.exp(-16 * factor))
    assert (np.abs(lse - want) <= 2.0 ** -17).all(), np.abs(lse - want).max()


@pytest.mark.parametrize("lens,prefix,Hq,Hkv,D,bs,window,sinks,hot", [
    # the hot key in either half of a tile, in odd and even tiles, among those that all rows see; sequences enough
    # for chains of several tiles
    ([40] * 20, [900] * 20, 16, 8, 128, 16, 0, 0, 300),
    ([40] * 20, [900] * 20, 16, 8, 128, 16, 0, 0, 850),
    ([40] * 20, [900] * 20, 16, 8, 64, 16, 0, 0, 300),
    ([40] * 20, [900] * 20, 16, 8, 64, 64, 0, 0, 600),
    ([1], [2900], 8, 1, 128, 16, 0, 0, 2850),                      # cut chains
    ([1, 1], [2900, 2900], 16, 2, 64, 16, 0, 0, 700),
    ([300, 300], [300, 700], 128, 8, 64, 16, 0, 0, 280),           # pairs of row tiles
    ([100] * 20, [1500] * 20, 16, 8, 128, 16, 700, 4, 1400),
    ([100] * 20, [1500] * 20, 16, 8, 64, 16, 700, 4, 1400),
])
def test_a_chunk_s_hot_key(lens, prefix, Hq, Hkv, D, bs, window, sinks, hot):
    c = Chunk(lens, prefix, Hq, Hkv, D, bs, window, sinks, seed=D + hot)
    g = np.random.default_rng(hot)
    factor = (1 + g.integers(8, 56, c.T) / 128.0)  # 17/16 .. 1.43: logits of 17 to 22.9, seven bits after the point
    c.q[:] = bits(factor)[:, None, None]
    seen = c.k != 0x7FC0
    c.k[seen], c.v[seen] = 0, cold(int(seen.sum()), hot)
    for b in range(len(lens)):
        c.k[c.table[b, hot // bs], :, hot % bs] = bits(16.0)
        c.v[c.table[b, hot // bs], :, hot % bs] = bits(HOT)
    t = c.tensors()
    import tree_attention_speculative_gb300 as ts
    p = c.params(t, scale=1.0 / D)
    ts.tree_chunk_attn_fwd(p, torch.zeros(ts.tree_chunk_attn_workspace_size(p), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert t["status"].cpu().tolist() == [0] * len(lens)
    n = int(c.cu[-1])
    pos = np.concatenate([np.arange(P, P + m) for P, m in zip(prefix, lens)])
    others = pos if not window else np.minimum(pos, window + sinks - 1)
    check(f64(t["out"])[:n], f64(t["lse"])[:n], factor[:n, None], others[:, None])


@pytest.mark.parametrize("D,N,prefix,hot", [(128, 26, 900, 700), (64, 26, 900, 700), (64, 40, 900, 850), (128, 200, 600, 0),
                                            (64, 200, 600, 0)])
def test_a_tree_s_hot_key(D, N, prefix, hot):
    """A key of the prefix, or (0) the root's."""
    from tree_attention_speculative_gb300.step import TreeVerifyStep
    B, window = 20, 4096
    c = W.build_case("hot", 5, W.tree_chain(N), [prefix] * B, 16, 8, D, 16, True)
    factor = 1 + np.random.default_rng(D + hot).integers(8, 56, (B, N)) / 128.0
    c.q[:] = bits(factor)[..., None, None]
    c.k_cache[:], c.k_tree[:] = 0, 0
    c.v_cache[:], c.v_tree[:] = cold(c.v_cache.shape, 1), cold(c.v_tree.shape, 2)
    for b in range(B):
        if hot:
            blk = c.block_table[b, hot // 16]
            c.k_cache[blk, :, hot % 16], c.v_cache[blk, :, hot % 16] = bits(16.0), bits(HOT)
        else:
            c.k_tree[b, 0], c.v_tree[b, 0] = bits(16.0), bits(HOT)
    t = to_dev(c)
    step = TreeVerifyStep(B, N, 16, 8, D, [prefix] * B, window=window, scale=1.0 / D)
    step.run(t["parent"], t["prefix_len"], t["q"], t["k_cache"], t["v_cache"], t["block_table"], t["k_tree"], t["v_tree"])
    torch.cuda.synchronize()
    assert step.status.cpu().tolist() == [0] * B
    check(f64(step.out), f64(step.lse), factor[..., None], (prefix + np.arange(N))[None, :, None])
