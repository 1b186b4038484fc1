"""The plans of chunk and windowed attention: which batches take pairs of row tiles, and what the queries refuse (no GPU
needed).  What tests/test_chunk_pairs_gpu.py and tests/test_chunk_pairs_cut_gpu.py run on pairs is planned so."""
import ctypes

import numpy as np
import pytest

from tests import test_chunk_pairs_cut_gpu, test_chunk_pairs_gpu
from tests.test_abi_host import _params, ts  # noqa: F401
from tests.test_prompt_host import _chunk, _i, _z


def plan(ts, lens, prefix, Hq, Hkv, D, bs, window, sinks):  # noqa: F811
    cu, kv = np.concatenate(([0], np.cumsum(lens))).astype(np.int32), np.add(lens, prefix).astype(np.int32)
    T, B, pool = int(cu[-1]), len(lens), (4, Hkv, bs, D)
    return ts.tree_chunk_attn_plan(_chunk(ts, q=_z(T, Hq, D), out=_z(T, Hq, D), lse=None, status=None, k_cache=_z(*pool),
                                          v_cache=_z(*pool), block_table=_i(B, -(-int(kv.max()) // bs)), cu_len=_i(B + 1),
                                          kv_len=_i(B), cu_len_host=cu, kv_len_host=kv, window=window, sinks=sinks))


@pytest.mark.parametrize("case", test_chunk_pairs_gpu.CASES[:6])
def test_batches_that_take_pairs(ts, case):  # noqa: F811
    p = plan(ts, *case)
    assert p["pairs"] and (p["max_splits"] > 1) == (case[0] == [300])


@pytest.mark.parametrize("case", test_chunk_pairs_cut_gpu.CASES)
def test_windowed_chains_cut_in_pairs(ts, case):  # noqa: F811
    p = plan(ts, *case)
    assert p["pairs"] and p["max_splits"] > 1


@pytest.mark.parametrize("case", [([300], [4000], 32, 2, 64, 64, 3500, 4), ([40], [257], 16, 1, 64, 128, 0, 0),
                                  ([4096], [12288], 32, 8, 128, 16, 0, 0)])
def test_batches_that_do_not(ts, case):  # noqa: F811
    """Too few items; one row tile; heads of 128."""
    assert not plan(ts, *case)["pairs"]


@pytest.mark.parametrize("N,prefix,window,sinks", [(40, (0, 10, 300, 129, 600, 5, 77, 256, 400, 128), 100, 5),
                                                   (37, (0, 10, 300, 129, 600, 5, 77, 256, 400, 128), 20, 3), (130, (300, 0, 129, 500), 64, 0)])
def test_trees_that_take_pairs(ts, N, prefix, window, sinks):  # noqa: F811
    p = _params(ts, B=len(prefix), N=N, Hq=128, Hkv=8, D=64, P=prefix)
    assert ts.tree_attn_window_plan(p, window, sinks)["pairs"]


def test_the_queries_refuse_what_the_calls_do(ts):  # noqa: F811
    L, p = ts.lib(), _chunk(ts)
    assert L.tree_chunk_attn_plan(ctypes.byref(p), None, None, None) == 0
    assert L.tree_chunk_attn_plan(None, None, None, None) == -1
    p.D = 96
    assert L.tree_chunk_attn_plan(ctypes.byref(p), None, None, None) == -4
    t = _params(ts)
    assert L.tree_attn_window_plan(ctypes.byref(t), 8, 0, None, None, None) == 0
    assert L.tree_attn_window_plan(ctypes.byref(t), 0, 0, None, None, None) == -2
