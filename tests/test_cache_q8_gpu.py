"""GPU parity of the 8-bit cache writers with the oracle: codes, scale bytes and
lengths are bit-exact, and nothing else in the pools changes."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_attention_speculative_gb300 import _build
    _build.build()


def _values(seed, shape):
    """bf16 rows over many magnitudes, with zero rows, zeros, subnormals, infinities and NaNs among them."""
    g = np.random.default_rng(seed)
    x = g.standard_normal(shape).astype(np.float32) * np.exp2(g.integers(-40, 40, shape[:-1] + (1,))).astype(np.float32)
    bits = W.bf16_bits(x)
    flat = bits.reshape(-1, shape[-1])
    n = len(flat)
    flat[g.integers(0, n, 1 + n // 16)] = 0
    flat[g.integers(0, n), 3] = 0x7F80            # +inf
    flat[g.integers(0, n), 5] = 0xFF80            # -inf
    flat[g.integers(0, n), 7] = 0x7FC0            # NaN
    flat[g.integers(0, n)] = 0x7FC0               # all NaN
    flat[g.integers(0, n)] = g.integers(0, 0x80, shape[-1])   # bf16 subnormals
    flat[g.integers(0, n), :2] = (0x7F7F, 0x43E0)  # largest finite; 448
    return bits


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _bf(bits):
    return _dev(bits.view(np.int16)).view(torch.bfloat16)


def _pool(nblk, Hkv, bs, D, seed=0):
    g = np.random.default_rng(seed)
    return (g.integers(0, 256, (nblk, Hkv, bs, D), np.uint8), g.integers(0, 256, (nblk, Hkv, bs, D), np.uint8),
            g.integers(0, 256, (nblk, Hkv, bs, 2), np.uint8))


def _table(need, nblk, seed):
    order = np.random.default_rng(seed).permutation(nblk)
    t = np.full((len(need), max(1, max(need))), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t


def _put(pool, table, b, t, k, v):
    """Row t of sequence b becomes k, v [Hkv, D] bf16 bits."""
    kc, vc, sc = pool
    bs = kc.shape[2]
    blk = table[b, t // bs]
    for x, c, w in ((k, kc, 0), (v, vc, 1)):
        codes, s = oracle.cache_q8.quantise(oracle.attention.bf16_to_f64(x))
        c[blk, :, t % bs], sc[blk, :, t % bs, w] = codes, s


APPENDS = [
    # lens, prefix, Hkv, D, bs
    ([1], [0], 1, 64, 16),
    ([1] * 9, [0, 1, 15, 16, 17, 100, 127, 128, 3], 8, 128, 16),
    ([0, 5, 0, 0, 33, 1, 0], [7, 3, 0, 48, 47, 0, 9], 2, 128, 48),
    ([300, 17], [5, 250], 3, 64, 144),
    ([129, 1, 64], [0, 63, 1], 5, 128, 64),
    ([0, 0], [4, 0], 2, 64, 16),
]


@pytest.mark.parametrize("lens,prefix,Hkv,D,bs", APPENDS)
@pytest.mark.parametrize("fused", [False, True])
def test_append_matches_oracle(lens, prefix, Hkv, D, bs, fused):
    import tree_attention_speculative_gb300 as ts
    B, T = len(lens), sum(lens)
    seed = T + D
    x = _values(seed, (T + 3, 2 * Hkv, D))  # three rows behind the last sequence
    k, v = x[:, :Hkv], x[:, Hkv:]
    need = [-(-(p + n) // bs) for p, n in zip(prefix, lens)]
    nblk = sum(need) + 2
    table, pool = _table(need, nblk, seed), _pool(nblk, Hkv, bs, D, seed)
    kd, vd, sd = (_dev(p) for p in pool)
    xd = _bf(x)
    kin, vin = xd[:, :Hkv], xd[:, Hkv:]
    if not fused:
        kin, vin = kin.contiguous(), vin.contiguous()
    cu = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
    new_len = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    status = torch.zeros(B, dtype=torch.int32, device="cuda")
    ts.tree_cache_append_q8(kin, vin, _dev(cu), _dev(np.array(prefix, np.int32)), kd.view(torch.float8_e4m3fn),
                            vd.view(torch.float8_e4m3fn), sd, _dev(table), new_len, status)
    for b in range(B):
        for i in range(lens[b]):
            _put(pool, table, b, prefix[b] + i, k[cu[b] + i], v[cu[b] + i])
    for got, want in zip((kd, vd, sd), pool):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    assert new_len.cpu().tolist() == [p + n for p, n in zip(prefix, lens)]
    assert status.cpu().tolist() == [0] * B


def test_append_many_rows():
    """Enough rows for the wide CTAs, compared through torch's own cast."""
    import tree_attention_speculative_gb300 as ts
    B, Hkv, D, bs = 5, 8, 128, 16
    lens = [1000, 1, 4099, 2500, 3333]
    T = sum(lens)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(T, Hkv, D, device="cuda", generator=g).bfloat16() for _ in range(2))
    need = [-(-n // bs) for n in lens]
    table = _dev(_table(need, sum(need), 3))
    pool = torch.zeros(2, sum(need), Hkv, bs, D, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(sum(need), Hkv, bs, 2, dtype=torch.uint8, device="cuda")
    cu = _dev(np.concatenate(([0], np.cumsum(lens))).astype(np.int32))
    zero, new_len = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    ts.tree_cache_append_q8(k, v, cu, zero, pool[0], pool[1], sc, table, new_len)
    assert new_len.cpu().tolist() == lens
    for w, x in enumerate((k, v)):
        top = x.float().abs().amax(-1)
        e = torch.frexp(top)[1] - 9 + (torch.frexp(top)[0] > 0.875) + 127
        codes = (x.float() * ((254 - e) << 23).view(torch.float32)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        for b in range(B):
            t = torch.arange(lens[b], device="cuda")
            blk = table[b].long()[t // bs]
            rows = slice(int(cu[b]), int(cu[b + 1]))
            assert torch.equal(pool[w][blk, :, t % bs], codes[rows])
            assert torch.equal(sc[blk, :, t % bs, w], e[rows].to(torch.uint8))


def test_append_reports_bad_sequences():
    """A failed sequence, a missing block, a table too short, cu_len out of order and a
    prefix past the limit keep their length; the others are written in full."""
    import tree_attention_speculative_gb300 as ts
    Hkv, D, bs = 2, 64, 16
    lens, prefix = [4, 20, 20, 3, 0, 5], [0, 10, 30, 2 ** 30, -1, 3]
    T = sum(lens)
    x = _values(5, (T, 2 * Hkv, D))
    table = np.array([[0, -1], [1, 2], [3, 4], [5, 5], [5, 5], [6, -1]], np.int32)
    table[1, 1] = 99          # outside the pool; sequence 2 ends past the table (50 tokens, 2 blocks)
    pool = _pool(8, Hkv, bs, D)
    kd, vd, sd = (_dev(p) for p in pool)
    cu = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
    new_len = torch.full((6,), -9, dtype=torch.int32, device="cuda")
    status = torch.tensor([0, 0, 0, 0, 0, -3], dtype=torch.int32, device="cuda")
    xd = _bf(x)
    ts.tree_cache_append_q8(xd[:, :Hkv], xd[:, Hkv:], _dev(cu), _dev(np.array(prefix, np.int32)), kd, vd, sd,
                            _dev(table), new_len, status)
    assert new_len.cpu().tolist() == [4, 10, 30, 2 ** 30, -1, 3]
    assert status.cpu().tolist() == [0, -5, -5, -2, -2, -3]
    for i in range(4):
        _put(pool, table, 0, i, x[i, :Hkv], x[i, Hkv:])
    got = kd.cpu().numpy()
    for blk in (0, 5, 6, 7):  # sequence 0's rows; nothing of sequences 3 to 5; the unused block
        np.testing.assert_array_equal(got[blk], pool[0][blk])
    # lengths out of order
    bad = np.array([0, 4, 2, T + 1, T + 1, T + 1, T + 1], np.int32)
    status.zero_()
    ts.tree_cache_append_q8(xd[:, :Hkv], xd[:, Hkv:], _dev(bad), torch.zeros(6, dtype=torch.int32, device="cuda"), kd,
                            vd, sd, _dev(np.zeros((6, 4), np.int32)), new_len, status)
    # (sequence 2 would take rows of sequence 0, which go to one of the two only, so neither counts)
    assert status.cpu().tolist() == [-2] * 6 and new_len.cpu().tolist() == [0] * 6


@pytest.mark.parametrize("cu,want", [
    ([0, 4, 2, 8, 9], [-2, -2, -2, 0]),     # rows 2 and 3 lie in sequences 0 and 2
    ([0, 2, 6, 5, 9], [0, -2, -2, -2]),     # row 5 in 1 and 3
    ([3, 0, 4, 8, 9], [-2, -2, 0, 0]),      # row 3 in sequence 1 and before sequence 0's end
    ([-1, 2, 4, 8, 9], [-2, 0, 0, 0]),
    ([0, 2, 4, 8, 10], [0, 0, 0, -2]),      # past the rows
    ([2, 2, 5, 5, 7], [0, 0, 0, 0]),        # rows of no sequence, and sequences without rows
])
def test_append_lengths_out_of_order(cu, want):
    """A sequence that reports nothing has every one of its rows; the others keep their length."""
    import tree_attention_speculative_gb300 as ts
    B, T, Hkv, D, bs = 4, 9, 2, 64, 16
    x = _values(6, (T, 2 * Hkv, D))
    xd = _bf(x)
    pool = _pool(B, Hkv, bs, D)
    kd, vd, sd = (_dev(p) for p in pool)
    table = np.arange(B, dtype=np.int32).reshape(B, 1)
    new = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    status = torch.zeros(B, dtype=torch.int32, device="cuda")
    ts.tree_cache_append_q8(xd[:, :Hkv], xd[:, Hkv:], _dev(np.array(cu, np.int32)),
                            torch.ones(B, dtype=torch.int32, device="cuda"), kd, vd, sd, _dev(table), new, status)
    assert status.cpu().tolist() == want
    assert new.cpu().tolist() == [1 + cu[b + 1] - cu[b] if want[b] == 0 else 1 for b in range(B)]
    got = [p.cpu().numpy() for p in (kd, vd, sd)]
    for b in range(B):
        if want[b] == 0:
            for t in range(cu[b], cu[b + 1]):
                _put(pool, table, b, 1 + t - cu[b], x[t, :Hkv], x[t, Hkv:])
            for p, q in zip(got, pool):
                np.testing.assert_array_equal(p[b], q[b])


def test_append_refuses_expanded_tokens():
    import tree_attention_speculative_gb300 as ts
    Hkv, D, bs = 2, 64, 16
    kd, vd, sd = (_dev(p) for p in _pool(2, Hkv, bs, D))
    x = _bf(_values(1, (5, Hkv, D)))
    new = torch.zeros(1, dtype=torch.int32, device="cuda")
    rest = (_dev(np.array([0, 5], np.int32)), torch.zeros(1, dtype=torch.int32, device="cuda"), kd, vd, sd,
            _dev(np.array([[0, 1]], np.int32)), new)
    for k, v in ((x[:1].expand(5, Hkv, D), x), (x, x[:1].expand(5, Hkv, D)), (x[:, :1].expand(5, Hkv, D), x)):
        with pytest.raises(ts.TreeSpecError):
            ts.tree_cache_append_q8(k, v, *rest)
    ts.tree_cache_append_q8(x, x, *rest)
    assert new.item() == 5


@pytest.mark.parametrize("Hkv,D,bs,depth", [(2, 128, 16, 7), (1, 64, 64, 3), (8, 128, 48, 19), (3, 64, 144, 0)])
def test_commit_matches_oracle(Hkv, D, bs, depth):
    import tree_attention_speculative_gb300 as ts
    B, N = 6, 33
    g = W.rng(bs, "commit-q8")
    prefix = np.array([0, 1, 15, 128, 300, 77], np.int32)
    L = np.minimum(np.array([0, 1, 2, 3, 7, 19], np.int32), depth)
    acc = np.full((B, depth + 1), -1, np.int32)
    for b in range(B):
        acc[b, :L[b] + 1] = np.sort(g.choice(N, L[b] + 1, replace=False))
    status = np.array([0, 0, -3, 0, 0, 0], np.int32)
    k, v = _values(1, (B, N, Hkv, D)), _values(2, (B, N, Hkv, D))
    need = [-(-(int(p) + depth + 1) // bs) for p in prefix]
    table, pool = _table(need, sum(need) + 1, 4), _pool(sum(need) + 1, Hkv, bs, D)
    bad = prefix[5] // bs
    table[5, bad] = -1          # sequence 5 commits nothing
    kd, vd, sd = (_dev(p) for p in pool)
    plen, st = _dev(prefix), _dev(status)
    ts.tree_commit_accepted_q8(_bf(k), _bf(v), _dev(acc), _dev(L), plen, kd, vd, sd, _dev(table), plen, st)
    for b in (0, 1, 3, 4):
        for d in range(L[b] + 1):
            _put(pool, table, b, int(prefix[b]) + d, k[b, acc[b, d]], v[b, acc[b, d]])
    for got, want in zip((kd, vd, sd), pool):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    want = prefix + L + 1
    want[[2, 5]] = prefix[[2, 5]]
    assert plen.cpu().tolist() == want.tolist() and st.cpu().tolist() == [0, 0, -3, 0, 0, -5]


def test_commit_ignores_lengths_and_nodes_out_of_range():
    import tree_attention_speculative_gb300 as ts
    B, N, Hkv, D, bs = 4, 3, 1, 64, 16
    pool = _pool(8, Hkv, bs, D)
    kd, vd, sd = (_dev(p) for p in pool)
    acc = np.array([[0, 1, 2, 2, 2], [0, 7, 0, 0, 0], [0, 0, 0, 0, 0], [0, 0, 0, 0, 0]], np.int32)
    L = np.array([3, 1, -1, 0], np.int32)   # longer than the tree; a node past it; negative; prefix past the limit
    plen = np.array([0, 5, 6, 2 ** 30 + 1], np.int32)
    st = torch.zeros(B, dtype=torch.int32, device="cuda")
    new = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    x = _bf(_values(1, (B, N, Hkv, D)))
    ts.tree_commit_accepted_q8(x, x, _dev(acc), _dev(L), _dev(plen), kd, vd, sd,
                               _dev(np.arange(8, dtype=np.int32).reshape(4, 2)), new, st)
    assert new.cpu().tolist() == plen.tolist() and st.cpu().tolist() == [0, -5, 0, 0]
    for got, want in zip((kd, vd, sd), pool):
        np.testing.assert_array_equal(got.cpu().numpy(), want)


def test_pool_rows_past_four_gigabytes():
    """Destinations whose byte offsets pass 32 bits."""
    import tree_attention_speculative_gb300 as ts
    Hkv, D, bs, nblk = 8, 128, 16, 300000     # 4.9 GB a pool
    kd, vd = (torch.empty(nblk, Hkv, bs, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    sd = torch.empty(nblk, Hkv, bs, 2, dtype=torch.uint8, device="cuda")
    x = _values(3, (20, 2 * Hkv, D))
    xd = _bf(x)
    table = np.array([[nblk - 1, nblk - 7]], np.int32)
    new = torch.empty(1, dtype=torch.int32, device="cuda")
    ts.tree_cache_append_q8(xd[:, :Hkv], xd[:, Hkv:], _dev(np.array([0, 20], np.int32)),
                            torch.zeros(1, dtype=torch.int32, device="cuda"), kd, vd, sd, _dev(table), new)
    for t in (0, 15, 16, 19):
        for w, (p, y) in enumerate(((kd, x[t, :Hkv]), (vd, x[t, Hkv:]))):
            codes, s = oracle.cache_q8.quantise(oracle.attention.bf16_to_f64(y))
            blk = table[0, t // bs]
            np.testing.assert_array_equal(p[blk, :, t % bs].cpu().numpy(), codes)
            np.testing.assert_array_equal(sd[blk, :, t % bs, w].cpu().numpy(), s)
