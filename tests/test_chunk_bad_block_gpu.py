"""Chunk attention of a batch in which one sequence's table names a block that is not there: block 0 is read in its place, for
that sequence alone; the other's keys and values lie elsewhere and its outputs are right."""
import numpy as np
import pytest
import torch

from tests.prompt_util import Chunk
from tests.test_chunk_attn_gpu import BAD_BLOCK, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_attention_speculative_gb300 import _build
    _build.build()


def free_block_0(c):
    """Block 0 becomes one that no sequence has, with zeros: what was there moves to the spare one."""
    spare = min(set(range(c.k.shape[0])) - set(c.table[c.table >= 0].tolist()))
    c.table = np.where(c.table == 0, spare, c.table)
    for pool in (c.k, c.v):
        pool[spare], pool[0] = pool[0].copy(), 0


@pytest.mark.parametrize("lens,prefix,Hq,Hkv,D,bs", [([20, 9], [100, 200], 4, 2, 128, 16), ([20, 9], [100, 200], 4, 2, 64, 16),
                                                     ([9, 20], [90, 1000], 4, 2, 128, 16), ([300, 130], [50, 400], 128, 8, 64, 16)])
@pytest.mark.parametrize("bad", [-1, "past"])
def test_the_other_sequence_is_right(lens, prefix, Hq, Hkv, D, bs, bad):
    c = Chunk(lens, prefix, Hq, Hkv, D, bs, seed=2)
    free_block_0(c)
    assert not (c.table == 0).any()
    t = c.tensors()
    t["table"][0, 3] = c.k.shape[0] if bad == "past" else bad
    run(c, t)
    assert t["status"].cpu().tolist() == [BAD_BLOCK, 0]
    c.table[0, 3] = 0
    c.check(t)  # (and the first one's, with block 0 in the bad one's place)
