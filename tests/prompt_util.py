"""Inputs and bounds of the prompt path's GPU tests."""
import numpy as np
import torch

import oracle
import workloads as W


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def bf(bits):
    return dev(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


NAN = 0x7FC0


def live_keys(p0, n, window, sinks):
    """Keys that some row at p0 .. p0 + n - 1 sees."""
    t = np.arange(p0 + n)
    if not window:
        return t
    return t[(t > p0 - window) | (t < sinks)]


class Chunk:
    """A ragged batch whose pools hold NaN everywhere but at the keys that some row sees, and whose table holds bad ids
    for blocks without such a key."""

    def __init__(self, lens, prefix, Hq, Hkv, D, bs, window=0, sinks=0, seed=0, extra_rows=2, hot=0.0, spare_blocks=1):
        self.lens, self.prefix, self.window, self.sinks, self.bs = lens, prefix, window, sinks, bs
        kv = [p + n for p, n in zip(prefix, lens)]
        table, nblk = W.paged_layout(W.rng(seed, "table"), np.array(kv, np.int32), bs, True)
        nblk += spare_blocks
        self.cu = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
        self.kv = np.array(kv, np.int32)
        T = int(self.cu[-1]) + extra_rows
        self.q = W.normal_bf16(seed, "q", (T, Hq, D))
        scale = np.where(W.rng(seed, "hot").random((nblk, Hkv, bs)) < hot, 8.0, 1.0) if hot else None
        k = W.normal_bf16(seed, "k", (nblk, Hkv, bs, D), scale)
        v = W.normal_bf16(seed, "v", (nblk, Hkv, bs, D))
        self.k, self.v = np.full_like(k, NAN), np.full_like(v, NAN)
        self.table = np.full(table.shape, -7, np.int32)
        for b, (p, n) in enumerate(zip(prefix, lens)):
            t = live_keys(p, n, window, sinks) if n else np.arange(0)
            blk = table[b, t // bs]
            self.table[b, t // bs] = blk
            for c, src in ((self.k, k), (self.v, v)):
                c[blk, :, t % bs] = src[blk, :, t % bs]
        self.T, self.Hq, self.Hkv, self.D = T, Hq, Hkv, D

    def tensors(self):
        t = dict(q=bf(self.q), k=bf(self.k), v=bf(self.v), table=dev(self.table), cu=dev(self.cu), kv=dev(self.kv))
        t["out"] = torch.full((self.T, self.Hq, self.D), 7.0, dtype=torch.bfloat16, device="cuda")
        t["lse"] = torch.full((self.T, self.Hq), 7.0, device="cuda")
        t["status"] = torch.zeros(len(self.lens), dtype=torch.int32, device="cuda")
        return t

    def params(self, t, scale=0.0, cu_host=None, kv_host=None):
        import tree_attention_speculative_gb300 as ts
        return ts.chunk_params(t["q"], t["k"], t["v"], t["table"], t["cu"], t["kv"],
                               self.cu if cu_host is None else cu_host, self.kv if kv_host is None else kv_host, t["out"],
                               t["lse"], t["status"], scale, self.window, self.sinks)

    def oracle(self, scale=0.0):
        a = (self.q, self.k, self.v, self.table, self.cu, self.kv)
        out, lse = oracle.window.chunk_attention(*a, scale=scale, window=self.window, sinks=self.sinks)
        mag, _ = oracle.window.chunk_attention(a[0], a[1], a[2] & 0x7FFF, *a[3:], scale=scale, window=self.window,
                                               sinks=self.sinks)
        return out, lse, mag

    def check(self, t, ref=None, scale=0.0, seqs=None):
        """out and lse of every sequence (or of some) against the oracle; the other rows as they were."""
        out, lse, mag = self.oracle(scale) if ref is None else ref
        got, got_lse = f64(t["out"]), f64(t["lse"])
        done = np.zeros(self.T, bool)
        for b in range(len(self.lens)) if seqs is None else seqs:
            done[self.cu[b]:self.cu[b + 1]] = True
        assert_rows(got[done], got_lse[done], out[done], lse[done], mag[done])
        if seqs is None:
            assert (got[~done] == 7).all() and (got_lse[~done] == 7).all()


def assert_rows(got, got_lse, out, lse, mag):
    """Each softmax weight is rounded to bf16 (2^-8 of it at most) and the output once more; `mag` is the output with the
    values' magnitudes.  Logits: 128 fp32 sums, off by up to 128 * 2^-24 of sum |q k| (below 64 here): 2^-11, which moves
    each weight by as much of it, and their normaliser.  lse: that and fp32's own steps."""
    tol = (2.0 ** -8 + 2.0 ** -10) * mag + 2.0 ** -8 * np.abs(out) + 1e-30
    bad = ~(np.abs(got - out) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], out[bad][:3])
    same = np.isneginf(lse)
    np.testing.assert_array_equal(np.isneginf(got_lse), same)
    assert (np.abs(got_lse - lse)[~same] <= 2.0 ** -10).all()
