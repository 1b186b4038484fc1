"""tree_chunk_attn_fwd against the fp64 oracle: ragged chunks, every group size, odd blocks, windows and sinks, over pools
that hold NaN wherever no row may look; graphs, many sequences, few CTAs and a wait that runs out."""
import numpy as np
import pytest
import torch

from tests.prompt_util import Chunk, dev, f64

pytestmark = pytest.mark.gpu

SHAPE, BAD_BLOCK, TIMEOUT = -2, -5, -6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_attention_speculative_gb300 import _build
    _build.build()


def run(c, t, p=None, ws=None, stream=None):
    import tree_attention_speculative_gb300 as ts
    p = c.params(t) if p is None else p
    if ws is None:
        ws = torch.zeros(ts.tree_chunk_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
    ts.tree_chunk_attn_fwd(p, ws, stream)
    torch.cuda.synchronize()
    assert (ws[:256] == 0).all()
    return ws


CASES = [
    # lens, prefix, Hq, Hkv, D, bs, window, sinks
    ([1], [0], 1, 1, 64, 16, 0, 0),
    ([1, 1, 1], [0, 16, 1000], 8, 2, 128, 16, 0, 0),
    ([5], [0], 2, 2, 64, 16, 0, 0),
    ([37, 0, 1, 130], [300, 5, 2047, 0], 8, 2, 128, 16, 0, 0),
    ([129, 64], [129, 640], 4, 2, 128, 32, 0, 0),          # rows past a tile, several row tiles
    ([40], [257], 16, 1, 64, 128, 0, 0),                    # 16 heads a group
    ([300], [7], 1, 1, 128, 48, 0, 0),                      # one head a group: 128 tokens a tile
    ([20, 3], [333, 150], 4, 2, 64, 80, 0, 0),
    ([9], [700], 16, 2, 128, 144, 0, 0),                    # 8 heads a group
    ([2], [6000], 8, 8, 128, 64, 0, 0),                     # a long chain, cut
    # windows
    ([1, 1, 1, 1], [0, 16, 1000, 3000], 8, 2, 128, 16, 64, 4),
    ([1], [5000], 4, 1, 64, 16, 1, 0),                      # the token alone
    ([130, 200], [700, 0], 4, 2, 64, 16, 100, 3),
    ([130], [2000], 2, 2, 128, 48, 129, 130),               # sinks past a tile
    ([17], [1500], 16, 1, 128, 144, 256, 0),
    ([50], [100], 4, 2, 64, 16, 1 << 30, 1 << 30),          # a window past everything
    ([33], [400], 4, 2, 128, 64, 20, 1 << 30),              # sinks past everything
    ([257], [1000], 1, 1, 64, 32, 128, 128),                # borders on tiles
    ([3], [128 * 9], 8, 1, 128, 128, 127, 1),
    ([1], [20000], 8, 1, 128, 64, 12000, 5),                # a long window, cut
]


@pytest.mark.parametrize("lens,prefix,Hq,Hkv,D,bs,window,sinks", CASES)
def test_matches_oracle(lens, prefix, Hq, Hkv, D, bs, window, sinks):
    c = Chunk(lens, prefix, Hq, Hkv, D, bs, window, sinks, seed=sum(lens) + D)
    t = c.tensors()
    run(c, t)
    assert t["status"].cpu().tolist() == [0] * len(lens)
    c.check(t)


def test_hot_keys_and_a_scale():
    c = Chunk([60, 1], [500, 900], 8, 2, 128, 16, seed=4, hot=0.05)
    t = c.tensors()
    run(c, t, c.params(t, scale=0.05))
    c.check(t, scale=0.05)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("levels", [
    [0, 40, 80, 120, 160, 200, 240], [240, 200, 160, 120, 80, 40, 0], [0, 0, 30, 30, 60, 0, 250], [-250, 250, -250, 0, -100, 9, 12],
    [5, 5, 5, 5, 5, 5, 5]])
def test_references_that_rise(D, levels):
    """Keys whose logits jump by tens to hundreds from tile to tile, whole numbers, so that logits are exact: the
    references are raised, some rows' more than once, and what came before is scaled down."""
    c = Chunk([70, 1], [7 * 128 - 70, 800], 4, 2, D, 16, seed=D)
    g = np.random.default_rng(1)
    one = np.uint16(0x3F80)
    c.q[:] = one
    for b in range(2):
        for t in range(int(c.kv[b])):
            for h in range(2):
                v = np.float32(levels[t // 128] + int(g.integers(0, 4)) - (h * 3 if t % 5 else 0))
                c.k[c.table[b, t // 16], h, t % 16] = np.uint16(v.view(np.uint32) >> 16)
    t = c.tensors()
    run(c, t, c.params(t, scale=1.0 / D))
    assert t["status"].cpu().tolist() == [0, 0]
    c.check(t, scale=1.0 / D)


def test_repeats_bit_for_bit_and_without_lse_or_status():
    import tree_attention_speculative_gb300 as ts
    c = Chunk([200, 1, 31], [900, 5000, 0], 8, 2, 128, 16, seed=6)
    t = c.tensors()
    ws = run(c, t)
    first, lse = t["out"].clone(), t["lse"].clone()
    for _ in range(3):
        t["out"].fill_(7.0)
        run(c, t, ws=ws)
        assert torch.equal(t["out"].view(torch.int16), first.view(torch.int16)) and torch.equal(t["lse"], lse)
    t["out"].fill_(7.0)
    p = ts.chunk_params(t["q"], t["k"], t["v"], t["table"], t["cu"], t["kv"], c.cu, c.kv, t["out"])
    run(c, t, p, ws)
    assert torch.equal(t["out"].view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("ctas", [1, 2, 3, 7])
@pytest.mark.parametrize("case", [3, 4, 12])
def test_many_items_through_few_ctas(ctas, case):
    import tree_attention_speculative_gb300 as ts
    c = Chunk(*CASES[case], seed=9)
    t = c.tensors()
    p = c.params(t)
    ws = torch.zeros(ts.tree_chunk_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
    ref = c.oracle()
    for _ in range(2):
        t["out"].fill_(7.0)
        t["lse"].fill_(7.0)
        ts.tree_chunk_attn_fwd_test(p, ws, ctas)
        torch.cuda.synchronize()
        assert (ws[:256] == 0).all()
        c.check(t, ref)
    assert t["status"].cpu().tolist() == [0] * len(c.lens)


@pytest.mark.parametrize("ctas,stall_tile", [(1, 0), (2, 1), (152, 0)])
def test_a_wait_that_runs_out(ctas, stall_tile):
    """The stalled sequence reports the timeout; those that report nothing are right; the next call is right."""
    import tree_attention_speculative_gb300 as ts
    c = Chunk([70, 33, 5], [300, 500, 40], 8, 2, 128, 16, seed=3)
    t = c.tensors()
    p = c.params(t)
    ws = torch.zeros(ts.tree_chunk_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
    ts.tree_chunk_attn_fwd_test(p, ws, ctas, stall_seq=1, stall_tile=stall_tile, wait_limit_us=3000)
    torch.cuda.synchronize()
    st = t["status"].cpu().tolist()
    assert st[1] == TIMEOUT and set(st) <= {0, TIMEOUT}
    if ctas == 152:
        assert st == [0, TIMEOUT, 0]
    assert (ws[:256] == 0).all()
    ref = c.oracle()
    c.check(t, ref, seqs=[b for b in range(3) if st[b] == 0])
    t = c.tensors()
    run(c, t, ws=ws)
    assert t["status"].cpu().tolist() == [0, 0, 0]
    c.check(t, ref)


def test_more_sequences_than_a_launch_takes():
    n = 300
    lens = [(b * 7) % 4 for b in range(n)]
    c = Chunk(lens, [(b * 37) % 90 for b in range(n)], 2, 1, 64, 16, seed=12)
    t = c.tensors()
    run(c, t)
    assert t["status"].cpu().tolist() == [0] * n
    c.check(t)


def test_a_bad_block_is_reported_and_the_others_are_right():
    c = Chunk([20, 9], [100, 200], 4, 2, 128, 16, seed=2)
    t = c.tensors()
    ref = c.oracle()
    t["table"][0, 3] = c.k.shape[0]
    t["k"][0], t["v"][0] = 0.0, 0.0  # read in its place
    ref_ok = 0 not in c.table[1, :-(-c.kv[1] // 16)]
    run(c, t)
    assert t["status"].cpu().tolist() == [BAD_BLOCK, 0]
    if ref_ok:
        c.check(t, ref, seqs=[1])


@pytest.mark.parametrize("change", ["cu_grown", "kv_short", "kv_past_table", "cu_past_T", "kv_negative"])
def test_device_lengths_that_are_not_the_plan_s(change):
    """The sequence reports TS_ERR_SHAPE, nothing of it is written, and the other one is right."""
    c = Chunk([20, 30], [100, 57], 4, 2, 128, 16, seed=7)
    t = c.tensors()
    p = c.params(t)
    if change == "cu_grown":
        t["cu"].copy_(dev(np.array([0, 20, 51], np.int32)))
    elif change == "kv_short":
        t["kv"].copy_(dev(np.array([120, 29], np.int32)))
    elif change == "kv_past_table":
        t["kv"].copy_(dev(np.array([120, c.table.shape[1] * 16 + 1], np.int32)))
    elif change == "cu_past_T":
        t["cu"].copy_(dev(np.array([0, 20, c.T + 1], np.int32)))
    else:
        t["kv"].copy_(dev(np.array([120, -5], np.int32)))
    run(c, t, p)
    assert t["status"].cpu().tolist() == [0, SHAPE]
    c.check(t, seqs=[0])
    assert (f64(t["out"])[20:] == 7).all()


def test_captured_calls_follow_growing_sequences_and_share_a_workspace():
    """Decoding in a graph: kv_len and the table grow between replays; two graphs on one workspace."""
    import tree_attention_speculative_gb300 as ts
    B = 3
    big = Chunk([1] * B, [700, 2000, 64], 8, 2, 128, 16, seed=21)
    t = big.tensors()
    start = np.array([300, 1200, 10], np.int32)
    p = big.params(t, kv_host=start)
    c2 = Chunk([33], [400], 8, 2, 128, 16, seed=22)
    t2 = c2.tensors()
    p2 = c2.params(t2)
    need = max(ts.tree_chunk_attn_workspace_size(p), ts.tree_chunk_attn_workspace_size(p2))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    ts.tree_chunk_attn_fwd(p, ws)
    ts.tree_chunk_attn_fwd(p2, ws)
    torch.cuda.synchronize()
    graphs = []
    for q in (p, p2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ts.tree_chunk_attn_fwd(q, ws)
        graphs.append(g)
    ref2 = c2.oracle()
    for kv in (start, start + 1, np.minimum(start * 2 - 7, big.kv), big.kv):  # (the tables end at big.kv)
        big.kv = np.array(kv, np.int32)
        t["kv"].copy_(dev(big.kv))
        for x in (t, t2):
            x["out"].fill_(7.0)
            x["lse"].fill_(7.0)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert t["status"].cpu().tolist() == [0] * B
        big.check(t)
        c2.check(t2, ref2)


def test_on_another_stream():
    c = Chunk([40, 1], [300, 1500], 8, 2, 128, 16, seed=30)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        t = c.tensors()
        run(c, t)
    c.check(t)
    t["out"].fill_(7.0)
    t["lse"].fill_(7.0)
    torch.cuda.synchronize()
    run(c, t, stream=s)
    c.check(t)


def test_a_cache_past_32_bits():
    """Pools of 2.2e9 elements: the highest blocks read as the same tokens in a small pool."""
    c = Chunk([5, 1], [300, 90], 8, 8, 128, 64, seed=31)
    t = c.tensors()
    run(c, t)
    want, lse = t["out"].clone(), t["lse"].clone()
    nblk = (2_200_000_000 // (8 * 64 * 128))
    small = c.k.shape[0]
    k, v = (torch.empty(nblk, 8, 64, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[nblk - small:], v[nblk - small:] = t["k"], t["v"]
    t.update(k=k, v=v, table=torch.where(t["table"] >= 0, t["table"] + (nblk - small), t["table"]))
    t["out"].fill_(7.0)
    run(c, t)
    assert t["status"].cpu().tolist() == [0, 0]
    assert torch.equal(t["out"].view(torch.int16), want.view(torch.int16)) and torch.equal(t["lse"], lse)


def test_no_tokens_at_all():
    import tree_attention_speculative_gb300 as ts
    c = Chunk([0, 0], [5, 40], 4, 2, 64, 16, extra_rows=0)
    t = c.tensors()
    p = c.params(t)
    ws = torch.zeros(max(256, ts.tree_chunk_attn_workspace_size(p)), dtype=torch.uint8, device="cuda")
    ts.tree_chunk_attn_fwd(p, ws)
    torch.cuda.synchronize()
    assert t["status"].cpu().tolist() == [0, 0]
