"""tree_cache_append_rope: turned queries and keys against the fp64 oracle, values and everything else exactly, both caches.

A turned value is within half a bf16 step of the exact one (2^-8 of it) plus the fp32 error of a pair, 2^-20 of its
length (sine and cosine to about 2^-22, two products and a sum)."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from tests.prompt_util import bf, dev, f64

pytestmark = pytest.mark.gpu

SHAPE, BAD_BLOCK = -2, -5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_attention_speculative_gb300 import _build
    _build.build()


class Batch:
    def __init__(self, lens, prefix, Hq, Hkv, D, bs, q8=False, fused=False, seed=0, extra=3):
        self.lens, self.prefix, self.Hq, self.Hkv, self.D, self.bs, self.q8 = lens, prefix, Hq, Hkv, D, bs, q8
        self.cu = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
        T = self.T = int(self.cu[-1]) + extra
        self.x = W.normal_bf16(seed, "x", (T, Hq + 2 * Hkv, D))
        need = [-(-(p + n) // bs) for p, n in zip(prefix, lens)]
        self.nblk = sum(need) + 2
        order = np.random.default_rng(seed).permutation(self.nblk)
        self.table = np.full((len(lens), max(1, max(need))), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        g = np.random.default_rng(seed + 1)
        shape = (self.nblk, Hkv, bs, D)
        self.pools = [g.integers(0, 256 if q8 else 60000, shape).astype(np.uint8 if q8 else np.uint16) for _ in range(2)]
        self.scales = g.integers(0, 256, (self.nblk, Hkv, bs, 2)).astype(np.uint8)
        xd = bf(self.x)
        self.q, self.k, self.v = xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:]
        if not fused:
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))
        self.kd, self.vd = ((dev(p).view(torch.float8_e4m3fn) if q8 else bf(p)) for p in self.pools)
        self.sd = dev(self.scales) if q8 else None
        self.q_out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.new_len = torch.full((len(lens),), -9, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(len(lens), dtype=torch.int32, device="cuda")

    def call(self, rope, with_q=True, **kw):
        import tree_attention_speculative_gb300 as ts
        a = dict(cu=dev(self.cu), prefix=dev(np.array(self.prefix, np.int32)), table=dev(self.table))
        a.update(kw)
        ts.tree_cache_append_rope(self.q if with_q else None, self.k, self.v, a["cu"], a["prefix"],
                                  self.q_out if with_q else None, self.kd, self.vd, a["table"], self.new_len, rope,
                                  self.status, self.sd)
        torch.cuda.synchronize()

    def pos(self):
        return np.concatenate([np.arange(p, p + n) for p, n in zip(self.prefix, self.lens)] + [np.zeros(0, int)]).astype(np.int64)

    def check(self, rope, with_q=True):
        n, D = int(self.cu[-1]), self.D
        pos = self.pos()
        x = oracle.attention.bf16_to_f64(self.x[:n])
        R = 0
        if rope is not None:
            R = rope.rotary_dim or D
            f = oracle.rope.frequencies(R, rope.theta, rope.scaling, rope.factor, rope.low_rot, rope.high_rot, rope.orig_len)
            turned = oracle.rope.rotate(x[:, :self.Hq + self.Hkv], pos, R, f, rope.interleaved, rope.mscale)
            ms = rope.mscale
        else:
            turned, ms = x[:, :self.Hq + self.Hkv], 1.0
        xs = x[:, :self.Hq + self.Hkv]
        length = ms * np.sqrt(2) * np.abs(xs[..., :max(R, 1)]).max(axis=-1, keepdims=True)
        tol = 2.0 ** -8 * np.abs(turned) + 2.0 ** -20 * length
        tol[..., R:] = 0
        got_q = f64(self.q_out)
        if with_q:
            assert (np.abs(got_q[:n] - turned[:, :self.Hq]) <= tol[:, :self.Hq]).all()
        assert (got_q[n if with_q else 0:] == 7).all()
        kt, ktol, v = turned[:, self.Hq:], tol[:, self.Hq:], self.x[:n, self.Hq + self.Hkv:]
        seq = np.repeat(np.arange(len(self.lens)), self.lens)
        blk, row = self.table[seq, pos // self.bs], pos % self.bs
        touched = np.zeros((self.nblk, self.bs), bool)
        touched[blk, row] = True
        if not self.q8:
            got_k, got_v = (t.view(torch.int16).cpu().numpy().view(np.uint16) for t in (self.kd, self.vd))
            assert (np.abs(oracle.attention.bf16_to_f64(got_k[blk, :, row]) - kt) <= ktol).all()
            np.testing.assert_array_equal(got_v[blk, :, row], v)
        else:
            got_k, got_v, got_s = (t.view(torch.uint8).cpu().numpy() for t in (self.kd, self.vd, self.sd))
            codes, s = oracle.cache_q8.quantise(oracle.attention.bf16_to_f64(v))
            np.testing.assert_array_equal(got_v[blk, :, row], codes)
            np.testing.assert_array_equal(got_s[blk, :, row, 1], s)
            # the key's scale: that of a row within its tolerance; its values: half a code step of the turned ones besides
            ks = got_s[blk, :, row, 0]
            _, lo = oracle.cache_q8.quantise(np.maximum(np.abs(kt) - ktol, 0))
            _, hi = oracle.cache_q8.quantise(np.abs(kt) + ktol)
            assert ((ks >= lo) & (ks <= hi)).all()
            val = oracle.cache_q8.values(got_k[blk, :, row], ks)
            step = 2.0 ** (ks.astype(np.float64)[..., None] - 127)
            assert (np.abs(val - kt) <= ktol + np.maximum(2.0 ** -4 * (np.abs(kt) + ktol), 2.0 ** -10 * step)).all()
            np.testing.assert_array_equal(got_s.transpose(0, 2, 1, 3)[~touched], self.scales.transpose(0, 2, 1, 3)[~touched])
        for got, was in ((got_k, self.pools[0]), (got_v, self.pools[1])):
            np.testing.assert_array_equal(got.transpose(0, 2, 1, 3)[~touched], was.transpose(0, 2, 1, 3)[~touched])
        assert self.new_len.cpu().tolist() == [p + m for p, m in zip(self.prefix, self.lens)]
        assert self.status.cpu().tolist() == [0] * len(self.lens)


BATCHES = [
    # lens, prefix, Hq, Hkv, D, bs
    ([1], [0], 1, 1, 64, 16),
    ([1] * 9, [0, 1, 15, 16, 17, 100, 127, 128, 3], 32, 8, 128, 16),
    ([0, 5, 0, 0, 33, 1, 0], [7, 3, 0, 48, 47, 0, 9], 6, 2, 128, 48),
    ([300, 17], [5, 250], 3, 3, 64, 144),
    ([1, 2], [(1 << 20) + 3, 70001], 4, 1, 128, 64),
    ([700], [9], 2, 1, 64, 16),
]
ROPES = [
    dict(),
    dict(theta=500000.0, scaling="bands", factor=8.0, orig_len=8192),
    dict(interleaved=True, rotary_dim=32, scaling="ntk", factor=16.0),
    dict(interleaved=True, mscale=1.2),
    dict(rotary_dim=20),                                     # no whole chunks
    dict(rotary_dim=10, interleaved=True, scaling="linear", factor=4.0),
    dict(rotary_dim=2),
    dict(rotary_dim=48),
]


@pytest.mark.parametrize("batch", range(len(BATCHES)))
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("rope", range(len(ROPES)))
def test_matches_oracle(batch, q8, rope):
    import tree_attention_speculative_gb300 as ts
    cfg = ts.RopeConfig(**ROPES[rope])
    b = Batch(*BATCHES[batch], q8=q8, fused=(batch + rope) % 2 == 0, seed=7 * batch + rope)
    b.call(cfg)
    b.check(cfg)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("rope", [None, 0])
def test_keys_and_values_alone(q8, rope):
    import tree_attention_speculative_gb300 as ts
    cfg = None if rope is None else ts.RopeConfig(**ROPES[rope])
    b = Batch([5, 0, 40], [30, 2, 100], 4, 2, 128, 16, q8=q8, fused=True, seed=50)
    b.call(cfg, with_q=False)
    b.check(cfg, with_q=False)


@pytest.mark.parametrize("q8", [False, True])
def test_agrees_with_the_separate_calls(q8):
    """tree_rope and then the append that there is (for the bf16 cache: the rows themselves)."""
    import tree_attention_speculative_gb300 as ts
    cfg = ts.RopeConfig(theta=500000.0)
    b = Batch([70, 3], [1000, 20], 8, 2, 128, 16, q8=q8, seed=60, extra=0)
    b.call(cfg)
    pos = dev(b.pos().astype(np.int32))[None]
    qo, ko = torch.empty_like(b.q)[None], torch.empty_like(b.k)[None]
    ts.tree_rope(b.q[None], b.k[None], pos, qo, ko, cfg)
    torch.cuda.synchronize()
    # the same angles and sums; a step of rounding at most where they are put together otherwise
    for got, want in ((f64(b.q_out), f64(qo[0])),):
        assert (np.abs(got - want) <= 2.0 ** -7 * np.abs(want)).all() and (got == want).mean() > 0.999
    if q8:
        kd, vd, sd = (dev(p) for p in (*b.pools, b.scales))
        new = torch.zeros(2, dtype=torch.int32, device="cuda")
        ts.tree_cache_append_q8(ko[0], b.v, dev(b.cu), dev(np.array(b.prefix, np.int32)), kd, vd, sd, dev(b.table), new)
        assert torch.equal(vd, b.vd.view(torch.uint8)) and torch.equal(new, b.new_len)
        assert (kd == b.kd.view(torch.uint8)).float().mean() > 0.999 and (sd == b.sd).float().mean() > 0.999


def test_rows_with_nan_and_infinity_in_the_8bit_cache():
    import tree_attention_speculative_gb300 as ts
    b = Batch([4], [0], 2, 1, 64, 16, q8=True, seed=61, extra=0)
    b.k[1, 0, 3] = float("nan")
    b.v[2, 0, 60] = float("inf")
    b.call(ts.RopeConfig())
    s = b.sd.cpu().numpy()[b.table[0, 0], 0]
    codes = b.kd.view(torch.uint8).cpu().numpy()[b.table[0, 0], 0]
    assert s[1, 0] == 255 and (codes[1] == 0x7F).all() and s[1, 1] != 255
    assert s[2, 1] == 247 and b.vd.view(torch.uint8).cpu().numpy()[b.table[0, 0], 0, 2, 60] == 0x7E


@pytest.mark.parametrize("fault,code", [("block", BAD_BLOCK), ("table", BAD_BLOCK), ("prefix", SHAPE), ("order", SHAPE),
                                        ("status", -3)])
def test_a_faulty_sequence_keeps_its_length(fault, code):
    import tree_attention_speculative_gb300 as ts
    b = Batch([20, 30], [100, 50], 4, 2, 128, 16, seed=62)
    kw = {}
    if fault == "block":
        b.table[1, 4] = b.nblk
    elif fault == "table":
        b.table = b.table[:, :4].copy()
        b.table[0, :] = b.table[0, :]
        kw["table"] = dev(b.table)
    elif fault == "prefix":
        kw["prefix"] = dev(np.array([100, -1], np.int32))
    elif fault == "order":
        kw["cu"] = dev(np.array([0, 20, 19], np.int32))
    else:
        b.status[1] = code
    was = b.kd.clone()
    b.call(ts.RopeConfig(), **kw)
    new, st = b.new_len.cpu().tolist(), b.status.cpu().tolist()
    assert st[1] == code and new[1] == (-1 if fault == "prefix" else 50)
    if fault == "table":
        return  # both sequences are longer than such a table's rows
    if fault != "order":
        assert (st[0], new[0]) == (0, 120)
    if fault in ("prefix", "status"):
        assert (f64(b.q_out)[20:] == 7).all()
        rows = b.table[1][b.table[1] >= 0]
        assert torch.equal(b.kd[rows].view(torch.int16), was[rows].view(torch.int16))  # (some are NaN)


def test_a_graph_replays_with_grown_lengths():
    import tree_attention_speculative_gb300 as ts
    cfg = ts.RopeConfig()
    b = Batch([1, 1], [30, 7], 4, 2, 128, 16, seed=63, extra=0)
    cu, table = dev(b.cu), dev(np.stack([np.arange(4), np.arange(4, 8)]).astype(np.int32) % b.nblk)
    prefix = dev(np.array(b.prefix, np.int32))

    def call():
        ts.tree_cache_append_rope(b.q, b.k, b.v, cu, prefix, b.q_out, b.kd, b.vd, table, b.new_len, cfg, b.status)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        prefix.copy_(b.new_len)
        g.replay()
        torch.cuda.synchronize()
    assert b.new_len.cpu().tolist() == [34, 11]
    f = oracle.rope.frequencies(128, cfg.theta)
    want = oracle.rope.rotate(f64(b.q), np.array([33, 10]), 128, f)
    assert np.abs(f64(b.q_out) - want).max() <= 2.0 ** -6


def test_a_pool_past_32_bits():
    import tree_attention_speculative_gb300 as ts
    b = Batch([3, 2], [60, 10], 8, 8, 128, 64, seed=64)
    cfg = ts.RopeConfig()
    b.call(cfg)
    b.check(cfg)
    nblk = 2_200_000_000 // (8 * 64 * 128)
    small_k, small_v = b.kd, b.vd
    b.kd, b.vd = (torch.empty(nblk, 8, 64, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    up = nblk - b.nblk
    b.kd[up:], b.vd[up:] = bf(b.pools[0]), bf(b.pools[1])
    b.call(cfg, table=dev(np.where(b.table >= 0, b.table + up, b.table)))
    assert torch.equal(b.kd[up:].view(torch.int16), small_k.view(torch.int16))
    assert torch.equal(b.vd[up:].view(torch.int16), small_v.view(torch.int16))


def test_no_tokens():
    import tree_attention_speculative_gb300 as ts
    b = Batch([0, 0], [4, 0], 2, 1, 64, 16, extra=0)
    b.call(ts.RopeConfig())
    assert b.new_len.cpu().tolist() == [4, 0] and b.status.cpu().tolist() == [0, 0]
