"""GPU parity of tree_attn_fwd_q8 with the fp64 oracle, given the values that the
quantised rows stand for.

Tolerance.  With A = sum p |v| / sum p (the same attention over |v|), an output
may be off by 2^-8 A for weights held in bf16, 2^-11 A for partials of a split
held in 16 bits with a row exponent, 2^-14 A for fp32 sums and the exponential,
and 2^-8 |out| for its own rounding to bf16.  The lse is fp32: a logit's error
is within 2^-18 of scale |q| |k| (the products' fp32 sums, and queries held to
2^-18 of their largest channel), and its own rounding 2^-18.
"""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from tests.gpu_util import SMALL, out_f64, to_dev
from tests.q8_util import codes_dev, quantised_pools, run_q8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_attention_speculative_gb300 import _build
    _build.build()


def _tree(g, kind, B, N):
    if kind == "random":
        return np.stack([W.tree_random_recursive(g, N) for _ in range(B)])
    if kind == "levels":
        return np.stack([W.tree_random_levels(g, N, 8) for _ in range(B)])
    return {"chain": W.tree_chain, "worked": lambda n: W.tree_worked_example(),
            "widths": lambda n: W.tree_from_widths([4, 3, 2, 1, 1])}[kind](N)


def _case(name, B, N, Hq, Hkv, D, plens, bs, tree, hot=0.0):
    g = W.rng(len(name), name)
    return W.build_case(name, 7, _tree(g, tree, B, N), plens, Hq=Hq, Hkv=Hkv, D=D, bs=bs,
                        permute=bs < max(max(plens), 1), hot_key_frac=hot)


def _abs_v(case):
    v = np.copy(case.v_cache), np.copy(case.v_tree)
    case.v_cache, case.v_tree = v[0] & 0x7FFF, v[1] & 0x7FFF
    A, _ = oracle.attention.tree_attention_case(case)
    case.v_cache, case.v_tree = v
    return A


def check(case, out, lse, ref=None, A=None):
    """out [B,N,Hq,D], lse [B,N,Hq] fp64 against the oracle on the case (its pools in bf16 bits)."""
    if ref is None:
        ref = oracle.attention.tree_attention_case(case)
    if A is None:
        A = _abs_v(case)
    tol = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -14) * A + 2.0 ** -8 * np.abs(ref[0]) + 2.0 ** -130
    bad = ~(np.abs(out - ref[0]) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, first {np.argwhere(bad)[:3].tolist()}, " \
                          f"worst {np.nanmax(np.abs(out - ref[0]) / tol)} of the tolerance"
    qn = np.sqrt((oracle.attention.bf16_to_f64(case.q) ** 2).sum(-1))
    kn = max(np.sqrt((oracle.attention.bf16_to_f64(x) ** 2).sum(-1)).max() for x in (case.k_cache, case.k_tree))
    off = np.abs(lse - ref[1])
    assert (off <= 2.0 ** -18 * (1 + np.abs(ref[1]) + case.scale * qn * kn)).all(), off.max()


def run_and_check(case):
    step, t = run_q8(case)
    assert step.status.cpu().tolist() == [0] * case.B
    check(case, out_f64(step), step.lse.double().cpu().numpy())
    return step, t


@pytest.mark.parametrize("spec", SMALL, ids=[s[0] for s in SMALL])
def test_small_elementwise(spec):
    run_and_check(_case(*spec))


MORE = [
    # one node: plain decoding; lengths around a tile and a block, and none
    ("decode", 9, 1, 8, 2, 128, [0, 1, 15, 16, 127, 128, 129, 255, 1000], 16, "chain"),
    ("decode_d64_g16", 5, 1, 16, 1, 64, [0, 1, 64, 129, 2000], 64, "chain"),
    ("decode_mha", 3, 1, 5, 5, 64, [77, 400, 1], 16, "chain"),
    # the rows of one warp of the tile, two fewer, one more, and half a warp with many units
    ("rows_32", 2, 8, 8, 2, 128, [3000, 1700], 16, "levels"),
    ("rows_30", 3, 15, 4, 2, 64, [2600, 0, 129], 48, "random"),
    ("rows_33", 2, 33, 2, 2, 128, [3000, 1700], 16, "levels"),
    ("rows_16_one_node", 40, 1, 16, 1, 128, [(211 * i) % 4000 for i in range(40)], 64, "chain"),
    # units of few rows of 128: trees of a few nodes; one row, two, three, eight, nine, sixteen, 17
    ("few_n4_g4", 5, 4, 8, 2, 128, [0, 77, 128, 1500, 4001], 16, "random"),
    ("few_n16_g1", 3, 16, 3, 3, 128, [2000, 5, 640], 48, "random"),
    ("few_n2_g4", 4, 2, 12, 3, 128, [3, 700, 129, 2222], 80, "chain"),
    ("few_n9_g1", 2, 9, 1, 1, 128, [9000, 128], 144, "levels"),
    ("few_n1_g1", 70, 1, 2, 2, 128, [(97 * i) % 700 for i in range(70)], 16, "chain"),
    ("few_long", 1, 3, 16, 4, 128, [40000], 64, "chain"),
    ("few_n2", 5, 2, 8, 2, 128, [0, 77, 128, 1500, 4001], 16, "chain"),
    ("few_n8_g1", 3, 8, 3, 3, 128, [2000, 5, 640], 48, "random"),
    ("few_n3_g1", 4, 3, 2, 2, 128, [3, 700, 129, 2222], 80, "random"),
    ("few_n1_g8", 40, 1, 16, 2, 128, [(211 * i) % 4000 for i in range(40)], 64, "chain"),
    ("few_n1_long", 1, 1, 8, 2, 128, [70001], 64, "chain"),
    ("n17_g1", 2, 17, 2, 2, 128, [1300, 257], 16, "random"),
    # two tree tiles; their second one word, one node, full
    ("n129", 2, 129, 2, 1, 128, [130, 0], 16, "random"),
    ("n256_d128", 1, 256, 2, 2, 128, [700], 48, "levels"),
    ("n256_g16", 1, 256, 16, 1, 64, [333], 16, "random"),
    # three KV heads, ragged, many splits
    ("hkv3", 3, 20, 12, 3, 128, [5000, 129, 0], 32, "levels"),
    ("splits_many", 1, 8, 4, 1, 128, [9000], 16, "levels"),
    ("splits_d64", 2, 30, 4, 1, 64, [5000, 37], 80, "levels"),
    # more (sequence, split) pairs than one table of the order holds
    ("many_pairs", 300, 3, 2, 1, 64, [(37 * i) % 600 for i in range(300)], 16, "chain"),
]


@pytest.mark.parametrize("spec", MORE, ids=[s[0] for s in MORE])
def test_more_layouts(spec):
    run_and_check(_case(*spec))


def test_hot_keys_and_scales_of_many_sizes():
    """Hot keys move the running maximum; rows of very different magnitude (2^-30 .. 2^30 for
    the values) put their scales far apart, so sums and rescaling must follow them."""
    case = _case("hot", 2, 40, 8, 2, 128, [1500, 700], 16, "levels", hot=0.02)
    g = np.random.default_rng(1)
    shape = case.v_cache.shape[:3]
    e = g.integers(-30, 31, shape + (1,))
    case.v_cache = W.bf16_bits((oracle.attention.bf16_to_f64(case.v_cache) * 2.0 ** e).astype(np.float32))
    e = g.integers(-3, 2, shape + (1,))
    case.k_cache = W.bf16_bits((oracle.attention.bf16_to_f64(case.k_cache) * 2.0 ** e).astype(np.float32))
    run_and_check(case)


@pytest.mark.parametrize("N,Hq", [(1, 16), (4, 4), (13, 1), (1, 8), (2, 4), (7, 1), (1, 1)])
def test_few_rows_of_growing_logits(N, Hq):
    """Keys that grow along the prefix raise a row's reference again and again; hot keys and scales
    of many sizes; queries from tiny to large; the step from the tree to the prefix."""
    case = _case("growing", 3, N, Hq, 1, 128, [2900, 131, 900], 16, "chain", hot=0.02)
    g = W.rng(8, "growing")
    pos = np.zeros(case.k_cache.shape[:3])
    for b in range(3):
        for t in range(int(case.prefix_len[b])):
            pos[case.block_table[b, t // 16], :, t % 16] = t / 300.0
    k = oracle.attention.bf16_to_f64(case.k_cache) * 2.0 ** pos[..., None]
    case.k_cache = W.bf16_bits(k.astype(np.float32))
    q = oracle.attention.bf16_to_f64(case.q) * 2.0 ** g.integers(-20, 3, case.q.shape[:3] + (1,))
    case.q = W.bf16_bits(q.astype(np.float32))
    run_and_check(case)


def test_queries_of_many_sizes():
    """Channels of a query far apart in size, a zero query, and tiny and huge ones (the keys undo them)."""
    case = _case("qsizes", 2, 33, 4, 2, 128, [300, 511], 16, "random")
    g = np.random.default_rng(2)
    q = oracle.attention.bf16_to_f64(case.q) * 2.0 ** g.integers(-12, 1, case.q.shape)
    q[0, 3] = 0.0
    q[0, 5] *= 2.0 ** -100
    q[1, 7, 0] *= 2.0 ** 4
    case.q = W.bf16_bits(q.astype(np.float32))
    run_and_check(case)


def _raw(case, pools, mask=None, plen_dev=None, workspace=None, table=None, stream=None, lse=True):
    import tree_attention_speculative_gb300 as ts
    t = to_dev(case)
    kc, vc, sc = (codes_dev(pools[0]), codes_dev(pools[1]), torch.from_numpy(pools[2]).cuda())
    B, N, Wd = case.B, case.N, (case.N + 63) // 64
    if mask is None:
        mask = oracle.tree.build_ancestry(case.parent, case.prefix_len)[0]
    anc = torch.from_numpy(mask.view(np.int64)).cuda()
    out = torch.full((B, N, case.Hq, case.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    ls = torch.full((B, N, case.Hq), float("nan"), dtype=torch.float32, device="cuda")
    status = torch.zeros(B, dtype=torch.int32, device="cuda")
    plen = t["prefix_len"] if plen_dev is None else torch.tensor(plen_dev, dtype=torch.int32, device="cuda")
    tab = t["block_table"] if table is None else torch.from_numpy(table).cuda()
    p = ts.attn_params(t["q"], kc, vc, tab, plen, case.prefix_len, t["k_tree"], t["v_tree"], anc, None, out,
                       ls if lse else None, status)
    if workspace is None:
        workspace = torch.zeros(ts.tree_attn_q8_workspace_size(p), dtype=torch.uint8, device="cuda")
    call = lambda s=stream: ts.tree_attn_fwd_q8(p, sc, workspace, s)  # noqa: E731
    call.keep = (t, kc, vc, sc, anc, plen, tab, workspace)
    return call, out, ls, status, workspace


def test_every_code_and_scale_through_the_values():
    """One prefix token takes all the weight: the output is its V row, exactly."""
    scales = [8, 60, 120, 127, 134, 190, 247]
    codes = np.arange(256, dtype=np.uint8).reshape(2, 128)
    codes = np.where((codes & 0x7F) == 0x7F, 0, codes)
    B = 2 * len(scales)
    case = W.build_case("codes", 3, W.tree_chain(1), [1] * B, Hq=1, Hkv=1, D=128, bs=16, permute=False)
    case.q[:], case.k_tree[:] = 0x3F80, 0xC1A0          # 1.0 and -20: logits of -226 for the node itself
    pools = [np.full(case.k_cache.shape, 0x7F, np.uint8), np.full(case.v_cache.shape, 0x7F, np.uint8),
             np.full(case.v_cache.shape[:3] + (2,), 255, np.uint8)]   # NaN and infinity behind the prefix
    want = np.empty((B, 128))
    for b in range(B):
        blk = case.block_table[b, 0]
        pools[0][blk, 0, 0], pools[1][blk, 0, 0] = 0x38, codes[b % 2]  # keys of 1.0
        pools[2][blk, 0, 0] = 127, scales[b // 2]
        want[b] = oracle.cache_q8.values(codes[b % 2][None], np.array([scales[b // 2]], np.uint8))[0]
    call, out, lse, status, _ = _raw(case, pools)
    call()
    # as bf16, which ends at 255 * 2^120: codes of 256 and more at the largest scale are infinite
    want = np.where(np.abs(want) > 255 * 2.0 ** 120, np.copysign(np.inf, want), want)
    np.testing.assert_array_equal(out.double().cpu().numpy()[:, 0, 0], want)
    assert status.cpu().tolist() == [0] * B


def test_every_code_through_the_keys():
    """No node is visible and one prefix token is: the lse is its logit."""
    codes = [c for c in range(256) if (c & 0x7F) != 0x7F]
    B = len(codes)
    case = W.build_case("kcodes", 3, W.tree_chain(1), [1] * B, Hq=1, Hkv=1, D=64, bs=16, permute=False)
    case.q[:] = 0
    case.q[:, 0, 0, 5] = 0x3FB5      # 1.4140625
    pools = [np.zeros(case.k_cache.shape, np.uint8), np.zeros(case.v_cache.shape, np.uint8),
             np.full(case.v_cache.shape[:3] + (2,), 127, np.uint8)]
    s = np.array([100 + b % 30 for b in range(B)], np.uint8)
    for b, c in enumerate(codes):
        blk = case.block_table[b, 0]
        pools[0][blk, 0, 0, 5], pools[2][blk, 0, 0, 0] = c, s[b]
    call, out, lse, status, _ = _raw(case, pools, mask=np.zeros((B, 1, 1), np.uint64))
    call()
    want = oracle.cache_q8.E4M3[codes] * 2.0 ** (s.astype(float) - 127) * 1.4140625 / 8
    np.testing.assert_allclose(lse.double().cpu().numpy()[:, 0, 0], want, rtol=2.0 ** -18, atol=1e-30)
    assert (out == 0).all()


@pytest.mark.parametrize("N,hidden", [(70, [0, 3, 64, 69]), (4, [1]), (1, [0])])
def test_rows_that_see_nothing(N, hidden):
    """Empty mask rows: the prefix alone; with no prefix, zeros and -inf; and the other rows as ever."""
    case = _case("empty", 3, N, 4, 2, 128, [0, 300, 5000], 16, "random")
    pools = quantised_pools(case)
    mask = oracle.tree.build_ancestry(case.parent, case.prefix_len)[0].copy()
    mask[:, hidden] = 0
    call, out, lse, status, _ = _raw(case, pools, mask=mask)
    call()
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    ref, A = oracle.attention.tree_attention_case(case), _abs_v(case)
    assert (got[0, hidden] == 0).all() and np.isneginf(gl[0, hidden]).all()
    for b in (1, 2):
        P = int(case.prefix_len[b])
        for h in range(case.Hq):
            rows = oracle.attention.bf16_to_f64(case.q[b, hidden, h])
            kv = [oracle.attention.prefix_kv(x, case.block_table, b, h // 2, P, case.bs) for x in (case.k_cache, case.v_cache)]
            see = np.ones((len(hidden), P), bool)
            ref[0][b, hidden, h], ref[1][b, hidden, h] = oracle.attention.attend_rows(rows, *kv, see, case.scale)
            A[b, hidden, h], _ = oracle.attention.attend_rows(rows, kv[0], np.abs(kv[1]), see, case.scale)
    got[0, hidden], gl[0, hidden] = ref[0][0, hidden], ref[1][0, hidden]
    check(case, got, gl, ref, A)


@pytest.mark.parametrize("N", [12, 2])
def test_garbage_behind_the_prefix_and_unused_table_entries(N):
    """NaN codes and scale bytes of 255 in every row past the prefix, table entries of -1 past its blocks."""
    case = _case("garbage", 4, N, 4, 1, 128, [0, 5, 130, 777], 48, "levels" if N > 2 else "chain")
    kc, vc, sc = quantised_pools(case)
    used = np.zeros(kc.shape[:1] + kc.shape[2:3], bool)
    table = np.full((4, case.block_table.shape[1] + 3), -1, np.int32)
    for b, P in enumerate(case.prefix_len):
        n = -(-int(P) // 48)
        table[b, :n] = case.block_table[b, :n]
        for t in range(P):
            used[case.block_table[b, t // 48], t % 48] = True
    blk, row = np.nonzero(~used)
    kc[blk, :, row], vc[blk, :, row], sc[blk, :, row] = 0x7F, 0xFF, 255
    call, out, lse, status, _ = _raw(case, (kc, vc, sc), table=table)
    call()
    assert status.cpu().tolist() == [0] * 4
    check(case, out.double().cpu().numpy(), lse.double().cpu().numpy())


@pytest.mark.parametrize("N", [10, 3])
def test_bad_blocks_and_long_device_prefixes_are_reported(N):
    """The other sequences are right; nothing is read outside the pool."""
    case = _case("report", 4, N, 4, 2, 128, [200, 300, 400, 100], 16, "levels" if N > 3 else "chain")
    pools = quantised_pools(case)
    table = case.block_table.copy()
    table[1, 3], table[1, 18] = 10 ** 6, -4
    call, out, lse, status, ws = _raw(case, pools, table=table, plen_dev=[200, 300, 10 ** 8, 100], lse=False)
    call()
    assert status.cpu().tolist() == [0, -5, -2, 0]
    got = out.double().cpu().numpy()
    ref, A = oracle.attention.tree_attention_case(case), _abs_v(case)
    for b in (0, 3):
        tol = (2.0 ** -8 + 2.0 ** -10) * A[b] + 2.0 ** -8 * np.abs(ref[0][b])
        assert (np.abs(got[b] - ref[0][b]) <= tol).all()
    call()   # the workspace is as it was
    torch.cuda.synchronize()
    assert torch.equal(out[0], torch.from_numpy(got[0]).cuda().bfloat16())
    assert (ws[:256] == 0).all()


def test_repeats_bit_for_bit_and_through_graphs_that_share_a_workspace():
    import tree_attention_speculative_gb300 as ts  # noqa: F401
    cases = [_case("graph", 3, 26, 8, 2, 128, [3000, 640, 17], 16, "widths"),
             _case("graph2", 2, 5, 4, 1, 64, [2000, 100], 64, "worked"),
             _case("graph3", 3, 1, 8, 2, 128, [4000, 9, 2222], 16, "chain")]
    need = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    calls = [_raw(c, quantised_pools(c), workspace=need) for c in cases]
    side = torch.cuda.Stream()
    want = []
    side.wait_stream(torch.cuda.current_stream())
    for c in calls:
        c[0](side)
        side.synchronize()
        want.append((c[1].clone(), c[2].clone()))
    for case, (o, l) in zip(cases, want):
        check(case, o.double().cpu().numpy(), l.double().cpu().numpy())
    graphs = []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c[0](None)
            c[0](None)
        graphs.append(g)
    for _ in range(3):
        for c in calls:
            c[1].fill_(7)
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for c, (o, l) in zip(calls, want):
        assert torch.equal(c[1], o) and torch.equal(c[2], l)


def test_pool_offsets_past_four_gigabytes():
    case = _case("far", 1, 9, 8, 8, 128, [200], 16, "levels")
    kc, vc, sc = quantised_pools(case)
    nblk = 300000     # 4.9 GB a pool
    big = [torch.empty(nblk, 8, 16, 128, dtype=torch.uint8, device="cuda") for _ in range(2)]
    bs = torch.empty(nblk, 8, 16, 2, dtype=torch.uint8, device="cuda")
    table = np.array([[nblk - 1 - 3 * i for i in range(13)]], np.int32)
    for i in range(13):
        old = case.block_table[0, i]
        for x, y in zip((*big, bs), (kc, vc, sc)):
            x[table[0, i]] = torch.from_numpy(y[old]).cuda()
    import tree_attention_speculative_gb300 as ts
    t = to_dev(case)
    anc = torch.from_numpy(oracle.tree.build_ancestry(case.parent, case.prefix_len)[0].view(np.int64)).cuda()
    out = torch.empty(1, 9, 8, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(1, 9, 8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tab = torch.from_numpy(table).cuda()  # held here: the parameter block keeps no tensor
    p = ts.attn_params(t["q"], *big, tab, t["prefix_len"], case.prefix_len, t["k_tree"],
                       t["v_tree"], anc, None, out, lse, status)
    ws = torch.zeros(ts.tree_attn_q8_workspace_size(p), dtype=torch.uint8, device="cuda")
    ts.tree_attn_fwd_q8(p, bs, ws)
    assert status.cpu().tolist() == [0]
    check(case, out.double().cpu().numpy(), lse.double().cpu().numpy())


def test_a_serving_loop():
    """Prompts appended, then three steps of ancestry, positions, attention, verify and commit on
    the 8-bit cache, against the same loop of the oracles."""
    import tree_attention_speculative_gb300 as ts
    from tree_attention_speculative_gb300.step import TreeVerifyStep
    from tests.test_cache_q8_gpu import _put
    B, N, Hq, Hkv, D, bs, V, depth = 3, 26, 8, 2, 128, 16, 200, 5
    cfg = ts.RopeConfig(theta=500000.0, scaling="bands", factor=8.0, orig_len=8192)
    freq = oracle.rope.frequencies(D, cfg.theta, "bands", 8.0, 1.0, 4.0, 8192)
    g = np.random.default_rng(4)
    plens = [0, 131, 40]
    T = sum(plens)
    bf = lambda x: torch.from_numpy(np.ascontiguousarray(x).view(np.int16)).cuda().view(torch.bfloat16)  # noqa: E731
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    nblk = 64
    pool = (np.zeros((nblk, Hkv, bs, D), np.uint8), np.zeros((nblk, Hkv, bs, D), np.uint8), np.zeros((nblk, Hkv, bs, 2), np.uint8))
    kd, vd, sd = torch.from_numpy(pool[0]).cuda(), torch.from_numpy(pool[1]).cuda(), torch.from_numpy(pool[2]).cuda()
    table = g.permutation(nblk)[:B * 20].reshape(B, 20).astype(np.int32)
    tab = i32(table)
    prompt = W.bf16_bits(g.standard_normal((T, 2 * Hkv, D)).astype(np.float32))
    cu = np.concatenate(([0], np.cumsum(plens)))
    pos = np.concatenate([np.arange(p) for p in plens])
    x = bf(prompt)
    k_rot = torch.empty(1, T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    ts.tree_rope(None, x[None, :, :Hkv], i32(pos[None]), None, k_rot, cfg)
    plen, new = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    status = torch.zeros(B, dtype=torch.int32, device="cuda")
    ts.tree_cache_append_q8(k_rot[0], x[:, Hkv:], i32(cu), plen, kd, vd, sd, tab, new, status)
    got_k = k_rot[0].view(torch.int16).cpu().numpy().view(np.uint16)
    for b in range(B):
        for i in range(plens[b]):
            _put(pool, table, b, i, got_k[cu[b] + i], prompt[cu[b] + i, Hkv:])
    plen, host = new, np.array(plens, np.int32)
    step = TreeVerifyStep(B, N, Hq, Hkv, D, host, vocab=V, max_depth=depth, rope=cfg)
    for turn in range(3):
        parent = np.stack([W.tree_from_widths([4, 3, 2, 1, 1])] * B)
        case = W.build_case(f"loop{turn}", turn, parent, host, Hq=Hq, Hkv=Hkv, D=D, bs=bs, permute=False, vocab=V,
                            plant_len=[turn, 5 - turn, 3])
        t = to_dev(case)
        step.prefix_len_host = host
        new = torch.empty_like(plen)
        step.run(t["parent"], plen, t["q"], kd, vd, tab, t["k_tree"], t["v_tree"], t["draft"], t["logits"], kv_scale=sd)
        step.commit(t["k_tree"], t["v_tree"], plen, kd, vd, tab, new, kv_scale=sd)
        # positions
        rot = {}
        for name, y in (("q", step.q_rot), ("k_tree", step.k_rot)):
            xs = oracle.attention.bf16_to_f64(getattr(case, name))
            rot[name] = y.view(torch.int16).cpu().numpy().view(np.uint16)
            at = host[:, None] + oracle.tree.build_ancestry(parent, host)[1]
            want = oracle.rope.rotate(xs.reshape(B * N, -1, D), at.reshape(-1), D, freq).reshape(xs.shape)
            assert (np.abs(oracle.attention.bf16_to_f64(rot[name]) - want) <= 2.0 ** -8 * np.abs(want) + 1e-5).all()
        # attention over the pool as it was before the commit
        case.q, case.k_tree, case.block_table = rot["q"], rot["k_tree"], table
        vals = [oracle.cache_q8.values(pool[w], pool[2][..., w]).astype(np.float32) for w in (0, 1)]
        case.k_cache, case.v_cache = W.bf16_bits(vals[0]), W.bf16_bits(vals[1])
        check(case, out_f64(step), step.lse.double().cpu().numpy())
        acc, L, _, _, _ = oracle.verify.verify_greedy(case.draft, case.logits, parent, depth)
        np.testing.assert_array_equal(step.accepted.cpu().numpy(), acc)
        for b in range(B):
            for d in range(L[b] + 1):
                _put(pool, table, b, int(host[b]) + d, rot["k_tree"][b, acc[b, d]], case.v_tree[b, acc[b, d]])
        for dev, want in zip((kd, vd, sd), pool):
            np.testing.assert_array_equal(dev.cpu().numpy(), want)
        host = (host + L + 1).astype(np.int32)
        assert new.cpu().tolist() == host.tolist() and step.status.cpu().tolist() == [0] * B
        plen = new


@pytest.mark.parametrize("N", [20, 2])
@pytest.mark.parametrize("host", [[3000, 100, 0], [900, 5000, 300]], ids=["grown", "mixed"])
def test_device_lengths_other_than_planned(host, N):
    """A captured launch keeps its plan while the device's lengths move, within the block table."""
    case = _case("moved", 3, N, 8, 2, 128, [2500, 2600, 700], 16, "levels" if N > 2 else "chain")
    pools = quantised_pools(case)
    true_len = case.prefix_len
    case.prefix_len = np.array(host, np.int32)
    width = 400
    table = np.full((3, width), -1, np.int32)
    table[:, :case.block_table.shape[1]] = case.block_table
    mask = oracle.tree.build_ancestry(case.parent, true_len)[0]
    call, out, lse, status, _ = _raw(case, pools, plen_dev=true_len.tolist(), table=table, mask=mask)
    call()
    assert status.cpu().tolist() == [0] * 3
    case.prefix_len = true_len
    check(case, out.double().cpu().numpy(), lse.double().cpu().numpy())


# (these lengths plan as short runs, so a segment has few tiles to stall before)
@pytest.mark.parametrize("N,stall_tile", [(26, 0), (26, 1), (26, 2), (3, 0), (3, 1), (2, 0), (2, 1), (2, 2)])
def test_a_wait_that_runs_out_is_reported(N, stall_tile):
    """One sequence's key stream stops: it reports TS_ERR_TIMEOUT, sequences that report nothing
    are right, and the next call on the same workspace is right everywhere."""
    import tree_attention_speculative_gb300 as ts
    case = _case("stall", 4, N, 8, 2, 128, [3000, 2000, 64, 1500], 16, "widths" if N == 26 else "chain")
    pools = quantised_pools(case)
    call, out, lse, status, ws = _raw(case, pools)
    t, kc, vc, sc, anc, plen, tab, _ = call.keep
    p = ts.attn_params(t["q"], kc, vc, tab, plen, case.prefix_len, t["k_tree"], t["v_tree"], anc, None, out, lse, status)
    ts.tree_attn_fwd_q8_stall_test(p, sc, ws, 1, stall_tile, 20000)
    torch.cuda.synchronize()
    st = status.cpu().tolist()
    assert st[1] == -6 and set(st) <= {0, -6}
    got = out.double().cpu().numpy()
    ref, A = oracle.attention.tree_attention_case(case), _abs_v(case)
    for b in range(4):
        if st[b] == 0:
            tol = (2.0 ** -8 + 2.0 ** -10) * A[b] + 2.0 ** -8 * np.abs(ref[0][b])
            assert (np.abs(got[b] - ref[0][b]) <= tol).all()
    status.zero_()
    call()
    assert status.cpu().tolist() == [0] * 4
    check(case, out.double().cpu().numpy(), lse.double().cpu().numpy(), ref, A)


@pytest.mark.parametrize("N", [5, 3])
def test_a_nan_row_reaches_its_sequence_and_head_alone(N):
    """V rows: every row that sees the token; K rows: the same, through the weights."""
    case = _case("nan", 3, N, 4, 2, 128, [300, 40, 70], 16, "worked" if N == 5 else "chain")
    pools = quantised_pools(case)
    for b, g, t, w in ((0, 0, 70, 1), (1, 1, 3, 0)):
        blk = case.block_table[b, t // 16]
        pools[w][blk, g, t % 16], pools[2][blk, g, t % 16, w] = 0x7F, 255
    call, out, lse, status, _ = _raw(case, pools)
    call()
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    nan = np.zeros(got.shape, bool)
    nan[0, :, :2] = nan[1, :, 2:] = True
    np.testing.assert_array_equal(np.isnan(got), nan)
    assert np.isnan(gl[1, :, 2:]).all() and not np.isnan(gl[0]).any()
    ref, A = oracle.attention.tree_attention_case(case), _abs_v(case)
    got[nan], gl[1, :, 2:] = ref[0][nan], ref[1][1, :, 2:]
    check(case, got, gl, ref, A)


@pytest.mark.parametrize("N,D", [(26, 128), (70, 64), (200, 128), (7, 128), (4, 128)])
def test_padding_and_hidden_keys_may_hold_anything(N, D):
    """Nodes no row sees hold NaN and infinities, a leaf's key too: only the leaf's own row shows it."""
    case = _case("padding", 3, N, 4, 2, D, [0, 300, 5000], 16, "random")
    pools = quantised_pools(case)
    mask = oracle.tree.build_ancestry(case.parent, case.prefix_len)[0].copy()
    parent = np.asarray(case.parent)
    pads, leaves = [], []
    for b in range(3):
        leaf = [n for n in range(N) if not (parent[b] == n).any()]
        pads.append(leaf[1:])
        leaves.append(leaf[0])
        mask[b, leaf[1:]] = 0
    clean = _raw(case, pools, mask=mask)
    clean[0]()
    junk = np.array([0x7FC0, 0x7F80, 0xFF80, 0xFFC1], np.uint16)
    for b in range(3):
        n = len(pads[b])
        case.v_tree[b, pads[b], :, 3] = junk[np.arange(n) % 4][:, None]
        case.k_tree[b, pads[b], :, D - 1] = junk[np.arange(n) % 4][:, None]
        case.k_tree[b, leaves[b], :, 5] = 0x7FC0
    dirty = _raw(case, pools, mask=mask)
    dirty[0]()
    for b in range(3):
        keep = [n for n in range(N) if n != leaves[b]]
        for x, y in ((clean[1], dirty[1]), (clean[2], dirty[2])):
            assert not torch.isnan(x[b]).any() and torch.equal(x[b, keep], y[b, keep])
            assert torch.isnan(y[b, leaves[b]]).all()


def test_step_keeps_a_captured_bf16_call_apart():
    """TreeVerifyStep reads either cache; the 8-bit call, which wants more workspace here, leaves
    the one that a captured bf16 call holds."""
    from tree_attention_speculative_gb300.step import TreeVerifyStep
    case = _case("apart", 1, 26, 32, 8, 128, [1024], 16, "widths")
    t = to_dev(case)
    step = TreeVerifyStep(1, 26, 32, 8, 128, case.prefix_len)
    args = (t["parent"], t["prefix_len"], t["q"])
    step.run(*args, t["k_cache"], t["v_cache"], t["block_table"], t["k_tree"], t["v_tree"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run(*args, t["k_cache"], t["v_cache"], t["block_table"], t["k_tree"], t["v_tree"])
    held, want = step.ws_attn, step.out.clone()
    pools = quantised_pools(case)
    kc, vc, sc = codes_dev(pools[0]), codes_dev(pools[1]), torch.from_numpy(pools[2]).cuda()
    for _ in range(2):
        step.run(*args, kc, vc, t["block_table"], t["k_tree"], t["v_tree"], kv_scale=sc)
        check(case, step.out.double().cpu().numpy(), step.lse.double().cpu().numpy())
        graph.replay()
        torch.cuda.synchronize()
        assert step.ws_attn is held and step.ws_attn_q8 is not held and torch.equal(step.out, want)
