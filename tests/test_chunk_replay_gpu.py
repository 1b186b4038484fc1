"""A captured chunk call whose sequences' rows change before it is replayed: fewer rows than planned are attended, more are
refused with TS_ERR_SHAPE, also where none were planned, and nothing of them is written."""
import numpy as np
import pytest
import torch

from tests.prompt_util import Chunk, bf, dev, f64

pytestmark = pytest.mark.gpu

SHAPE = -2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_attention_speculative_gb300 import _build
    _build.build()


MANY = [1, 0] * 299 + [0, 0]


@pytest.mark.parametrize("planned,now", [
    ([5, 0, 40], [5, 0, 40]), ([5, 0, 40], [2, 0, 17]), ([5, 0, 40], [0, 0, 0]), ([5, 0, 40], [6, 0, 39]),
    ([5, 0, 40], [5, 3, 37]), ([0, 0, 40], [0, 4, 30]), ([0, 0, 40], [2, 0, 30]), ([40, 0, 0, 0], [33, 0, 0, 7]),
    ([9, 0, 0, 3, 0, 7], [5, 2, 1, 3, 4, 0]),
    ([300, 0, 400, 0], [300, 2, 397, 1]),                                                # more items than SMs
    (MANY, [1, 0] * 100 + [0, 1] * 2 + [1, 0] * 196 + [0, 0, 0, 1]),                           # more sequences than a launch takes
])
@pytest.mark.parametrize("ctas", [None, 2])
def test_rows_that_changed(planned, now, ctas):
    import tree_attention_speculative_gb300 as ts
    B, T = len(planned), sum(planned)
    assert sum(now) <= T and len(now) == B
    total = [p + 30 + b * 13 % 300 for b, p in enumerate(planned)]
    first = Chunk(planned, [m - n for m, n in zip(total, planned)], 16, 8, 128, 16, seed=1)
    t = first.tensors()
    p = first.params(t)
    ws = torch.zeros(ts.tree_chunk_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
    call = (lambda: ts.tree_chunk_attn_fwd(p, ws)) if ctas is None else (lambda: ts.tree_chunk_attn_fwd_test(p, ws, ctas))
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    c = Chunk(now, [m - n for m, n in zip(total, now)], 16, 8, 128, 16, seed=1, extra_rows=T + 2 - sum(now))
    assert c.k.shape == first.k.shape
    for name, x in (("q", bf(c.q)), ("k", bf(c.k)), ("v", bf(c.v)), ("table", dev(c.table)), ("cu", dev(c.cu)), ("kv", dev(c.kv))):
        t[name].copy_(x)
    t["out"].fill_(7.0)
    t["lse"].fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    status = [SHAPE if n > m else 0 for n, m in zip(now, planned)]
    assert t["status"].cpu().tolist() == status and (ws[:256] == 0).all()
    live = [b for b in range(B) if status[b] == 0]
    c.check(t, seqs=live)
    left = np.ones(c.T, bool)
    for b in live:
        left[c.cu[b]:c.cu[b + 1]] = False
    assert (f64(t["out"])[left] == 7).all() and (f64(t["lse"])[left] == 7).all()
