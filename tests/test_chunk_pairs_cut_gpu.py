"""Chunk attention on pairs of row tiles whose chains of keys have a window and are cut: the tiles that the window or the sinks
end in, and the join of the parts, against the fp64 oracle, over pools that hold NaN wherever no row may look."""
import pytest
import torch

from tests.prompt_util import Chunk
from tests.test_chunk_attn_gpu import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_attention_speculative_gb300 import _build
    _build.build()


CASES = [
    # lens, prefix, Hq, Hkv, D, bs, window, sinks
    ([300], [4000], 32, 2, 64, 16, 3000, 200),      # sinks past a tile
    ([500], [9000], 16, 2, 64, 16, 6000, 4),
    ([600], [8000], 16, 1, 64, 16, 7000, 0),
    ([590, 3], [8000, 70], 16, 1, 64, 16, 7001, 129),  # a second sequence with one row tile
]


@pytest.mark.parametrize("lens,prefix,Hq,Hkv,D,bs,window,sinks", CASES)
def test_matches_oracle(lens, prefix, Hq, Hkv, D, bs, window, sinks):
    import tree_attention_speculative_gb300 as ts
    c = Chunk(lens, prefix, Hq, Hkv, D, bs, window, sinks, seed=sum(lens))
    t = c.tensors()
    p = c.params(t)
    plan = ts.tree_chunk_attn_plan(p)
    assert plan["pairs"] and plan["max_splits"] > 1
    ws = run(c, t, p)
    assert t["status"].cpu().tolist() == [0] * len(lens)
    c.check(t)
    first = t["out"].clone()
    t["out"].fill_(7.0)
    run(c, t, p, ws)
    assert torch.equal(t["out"].view(torch.int16), first.view(torch.int16))
