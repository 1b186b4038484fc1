"""Pools of the wrong width are refused before a pointer is passed on (no GPU needed): the
8-bit pools have the bf16 pools' shape and argument slots, and half their bytes."""
import numpy as np
import pytest
import torch

from tests.test_abi_host import ts  # noqa: F401

SHAPE = -2
B, N, HQ, HKV, D, BS, NBLK, MAXB = 3, 6, 4, 2, 64, 16, 9, 5


def _z(*s, dtype=torch.bfloat16):
    return torch.zeros(*s, dtype=dtype)


def _i(*s):
    return torch.zeros(*s, dtype=torch.int32)


def _pool(dtype):
    return _z(NBLK, HKV, BS, D, dtype=torch.uint8).view(dtype) if dtype.itemsize == 1 else _z(NBLK, HKV, BS, D, dtype=dtype)


def _attn_args(**kw):
    a = dict(q=_z(B, N, HQ, D), k_cache=_pool(torch.bfloat16), v_cache=_pool(torch.bfloat16), block_table=_i(B, MAXB),
             prefix_len=_i(B), prefix_len_host=np.zeros(B, np.int32), k_tree=_z(B, N, HKV, D), v_tree=_z(B, N, HKV, D),
             anc_mask=torch.zeros(B, N, 1, dtype=torch.int64), pos=_i(B, N), out=_z(B, N, HQ, D),
             lse=_z(B, N, HQ, dtype=torch.float32), status=_i(B))
    a.update(kw)
    return a


def _refused(ts, call):  # noqa: F811
    with pytest.raises(ts.TreeSpecError) as e:
        call()
    assert e.value.status == SHAPE


NARROW = [dict(k_cache=d, v_cache=d) for d in (torch.uint8, torch.float8_e4m3fn)] + \
         [dict(k_cache=torch.uint8), dict(v_cache=torch.float8_e4m3fn), dict(k_cache=torch.float32)]


@pytest.mark.parametrize("kw", NARROW)
def test_bf16_calls_refuse_pools_of_another_width(ts, kw):  # noqa: F811
    pools = {k: _pool(d) for k, d in kw.items()}
    p, ws = ts.attn_params(**_attn_args(**pools)), _z(1 << 20, dtype=torch.uint8)
    _refused(ts, lambda: ts.tree_attn_fwd(p, ws, 0))
    _refused(ts, lambda: ts.tree_attn_fwd_stall_test(p, ws, 0, 0, 1000, 0))
    _refused(ts, lambda: ts.tree_attn_fwd_ctas_test(p, ws, 1, stream=0))
    c = dict(k_cache=_pool(torch.bfloat16), v_cache=_pool(torch.bfloat16))
    c.update(pools)
    _refused(ts, lambda: ts.tree_commit_accepted(_z(B, N, HKV, D), _z(B, N, HKV, D), _i(B, 4), _i(B), _i(B), c["k_cache"],
                                                 c["v_cache"], _i(B, MAXB), _i(B), _i(B), 0))


def test_a_step_refuses_8bit_pools_without_their_scales(ts):  # noqa: F811
    from tree_attention_speculative_gb300.step import TreeVerifyStep
    step = TreeVerifyStep(B, N, HQ, HKV, D, np.zeros(B, np.int32), vocab=10, device="cpu")
    kc, vc, table, plen = _pool(torch.float8_e4m3fn), _pool(torch.float8_e4m3fn), _i(B, MAXB), _i(B)
    k, v = _z(B, N, HKV, D), _z(B, N, HKV, D)
    _refused(ts, lambda: step.attention(_z(B, N, HQ, D), kc, vc, table, plen, k, v, 0))
    _refused(ts, lambda: step.commit(k, v, plen, kc, vc, table, _i(B), 0))
