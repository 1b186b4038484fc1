"""Appends of a batch with sequences whose sizes are wrong: they report TS_ERR_SHAPE, keep their lengths, and nothing of them
is written, neither queries nor rows of the cache; the others are as they would be alone."""
import numpy as np
import pytest
import torch

from tests.prompt_util import dev, f64
from tests.test_append_rope_gpu import SHAPE, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_attention_speculative_gb300 import _build
    _build.build()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("lens,cu,faulty", [
    ([20, 30], [0, 20, 19], [0, 1]),                              # the second ends before it begins, inside the first
    ([20, 30], [0, 20, 54], [1]),                                 # past the last row (53)
    ([20, 30, 0, 10], [0, 20, 50, 45, 55], [1, 2, 3]),            # a boundary inside a neighbour
    ([20, 30, 0, 10], [0, 20, 50, 50, 64], [3]),
    ([5] * 300, [0] + [5 * (b + 1) for b in range(299)] + [1480], list(range(296, 300))),  # more sequences than threads
])
def test_nothing_of_a_faulty_sequence_is_written(lens, cu, faulty, q8):
    import tree_attention_speculative_gb300 as ts
    prefix = [100 + 3 * b % 50 for b in range(len(lens))]
    b = Batch(lens, prefix, 4, 2, 128, 16, q8=q8, seed=70)
    good, cfg = Batch(lens, prefix, 4, 2, 128, 16, q8=q8, seed=70), ts.RopeConfig()
    good.call(cfg)
    was = [t.view(torch.uint8).clone() for t in (b.kd, b.vd)]
    b.call(cfg, cu=dev(np.array(cu, np.int32)))
    assert b.status.cpu().tolist() == [SHAPE if s in faulty else 0 for s in range(len(lens))]
    assert b.new_len.cpu().tolist() == [p + (0 if s in faulty else n) for s, (p, n) in enumerate(zip(prefix, lens))]
    q, want = f64(b.q_out), f64(good.q_out)
    live = np.zeros(b.T, bool)
    for s, n in enumerate(lens):
        if s not in faulty:
            live[b.cu[s]:b.cu[s] + n] = True
        rows = dev(b.table[s][b.table[s] >= 0]).long()
        for got, old, new in zip((b.kd, b.vd), was, (good.kd, good.vd)):
            assert torch.equal(got.view(torch.uint8)[rows], old[rows] if s in faulty else new.view(torch.uint8)[rows])
    np.testing.assert_array_equal(q[live], want[live])
    assert (q[~live] == 7).all()
