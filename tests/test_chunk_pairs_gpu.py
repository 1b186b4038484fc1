"""Chunk and windowed attention where an item takes a pair of row tiles (heads of 64, more items than SMs or nearly so),
against the fp64 oracle, over pools that hold NaN wherever no row may look."""
import numpy as np
import pytest
import torch

from tests.prompt_util import Chunk, assert_rows, f64
from tests.test_attn_window_gpu import build
from tests.test_attn_window_gpu import run as run_tree
from tests.test_chunk_attn_gpu import TIMEOUT, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_attention_speculative_gb300 import _build
    _build.build()


CASES = [
    # lens, prefix, Hq, Hkv, D, bs, window, sinks
    ([300, 9, 1, 130], [50, 400, 600, 0], 128, 8, 64, 16, 0, 0),  # 8 tokens a tile: odd numbers of them, one, part of one
    ([300, 9, 1, 131], [50, 400, 600, 0], 128, 8, 64, 48, 0, 0),
    ([300, 9, 1, 130], [350, 400, 600, 0], 128, 8, 64, 16, 100, 5),
    ([300, 17, 0, 90], [777, 3, 0, 256], 128, 8, 64, 32, 128, 130),  # borders on tiles, sinks past one
    # one head a group: 128 tokens a tile
    ([300, 257, 513, 256, 31, 300, 400, 129, 300, 260], [0, 100, 5, 200, 40, 0, 3, 300, 20, 1], 8, 8, 64, 16, 0, 0),
    ([300], [4000], 32, 2, 64, 16, 0, 0),                            # cut chains
    ([300], [4000], 32, 2, 64, 64, 3500, 4),
]


@pytest.mark.parametrize("lens,prefix,Hq,Hkv,D,bs,window,sinks", CASES)
def test_matches_oracle(lens, prefix, Hq, Hkv, D, bs, window, sinks):
    c = Chunk(lens, prefix, Hq, Hkv, D, bs, window, sinks, seed=sum(lens) + bs)
    t = c.tensors()
    ws = run(c, t)
    assert t["status"].cpu().tolist() == [0] * len(lens)
    c.check(t)
    first = t["out"].clone()
    t["out"].fill_(7.0)
    run(c, t, ws=ws)
    assert torch.equal(t["out"].view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("levels", [[0, 40, 80, 120, 160, 200, 240], [0, 0, 30, 30, 60, 0, 250], [-250, 250, -250, 0, -100, 9, 12]])
def test_references_that_rise(levels):
    """Logits that jump by tens to hundreds from tile to tile, whole numbers, so that they are exact."""
    c = Chunk([70, 1, 70, 70], [7 * 128 - 70, 800, 826, 826], 128, 8, 64, 16, seed=3)
    g = np.random.default_rng(1)
    c.q[:] = np.uint16(0x3F80)
    for b in range(4):
        for t in range(int(c.kv[b])):
            v = np.float32(levels[t // 128] + g.integers(0, 4, 8) - (np.arange(8) * 3 if t % 5 else 0))
            c.k[c.table[b, t // 16], :, t % 16] = (v.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)[:, None]
    t = c.tensors()
    run(c, t, c.params(t, scale=1.0 / 64))
    assert t["status"].cpu().tolist() == [0] * 4
    c.check(t, scale=1.0 / 64)


@pytest.mark.parametrize("ctas", [1, 7])
def test_many_items_through_few_ctas(ctas):
    import tree_attention_speculative_gb300 as ts
    c = Chunk(*CASES[2], seed=9)
    t = c.tensors()
    p = c.params(t)
    ws = torch.zeros(ts.tree_chunk_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
    ts.tree_chunk_attn_fwd_test(p, ws, ctas)
    torch.cuda.synchronize()
    assert (ws[:256] == 0).all() and t["status"].cpu().tolist() == [0] * 4
    c.check(t)


@pytest.mark.parametrize("ctas,stall_tile", [(2, 0), (5, 1)])
def test_a_wait_that_runs_out(ctas, stall_tile):
    """The stalled sequence reports the timeout; those that report nothing are right; the next call is right."""
    import tree_attention_speculative_gb300 as ts
    c = Chunk([300, 40, 1, 130], [50, 400, 600, 0], 128, 8, 64, 16, seed=4)
    t = c.tensors()
    p = c.params(t)
    ws = torch.zeros(ts.tree_chunk_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
    ts.tree_chunk_attn_fwd_test(p, ws, ctas, stall_seq=1, stall_tile=stall_tile, wait_limit_us=3000)
    torch.cuda.synchronize()
    st = t["status"].cpu().tolist()
    assert st[1] == TIMEOUT and set(st) <= {0, TIMEOUT}
    assert (ws[:256] == 0).all()
    ref = c.oracle()
    c.check(t, ref, seqs=[b for b in range(4) if st[b] == 0])
    t = c.tensors()
    run(c, t, ws=ws)
    assert t["status"].cpu().tolist() == [0] * 4
    c.check(t, ref)


@pytest.mark.parametrize("N,kind,window,sinks", [(40, "random", 100, 5), (37, "chain", 20, 3), (130, "random", 64, 0)])
def test_trees(N, kind, window, sinks):
    prefix = [0, 10, 300, 129, 600, 5, 77, 256, 400, 128] if N < 100 else [300, 0, 129, 500]
    c, ref = build(N, kind, prefix, 128, 8, 64, 16, window, sinks, seed=N)
    step = run_tree(c, window, sinks)
    assert step.status.cpu().tolist() == [0] * c.B
    assert_rows(f64(step.out), f64(step.lse), *ref)
