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


def _q8_args(**kw):
    return _attn_args(**{**dict(k_cache=_pool(torch.float8_e4m3fn), v_cache=_pool(torch.float8_e4m3fn)), **kw})


def _q8_refused(ts, a, sc=None, ws=None):  # noqa: F811
    sc = _z(NBLK, HKV, BS, 2, dtype=torch.uint8) if sc is None else sc
    ws = _z(1 << 20, dtype=torch.uint8) if ws is None else ws
    _refused(ts, lambda: ts.tree_attn_fwd_q8(ts.attn_params(**a), sc, ws, 0))
    _refused(ts, lambda: ts.tree_attn_fwd_q8_stall_test(ts.attn_params(**a), sc, ws, 0, 0, 1000, 0))


@pytest.mark.parametrize("kw", [
    dict(v_cache=_z(NBLK - 1, HKV, BS, D, dtype=torch.uint8)), dict(v_cache=_z(NBLK, HKV, BS, 2 * D, dtype=torch.uint8)),
    dict(k_cache=_z(NBLK, BS, HKV, D, dtype=torch.uint8).transpose(1, 2)), dict(k_cache=_z(NBLK, HKV, BS, D // 2, dtype=torch.uint8)),
    dict(v_cache=_pool(torch.bfloat16)), dict(block_table=_i(B, MAXB).long()), dict(block_table=_i(B, 2 * MAXB)[:, ::2]),
    dict(block_table=_i(B - 1, MAXB)), dict(prefix_len=_i(B).long()), dict(prefix_len=_i(B - 1)),
    dict(prefix_len_host=np.zeros(B - 1, np.int32)), dict(q=_z(B, N, HQ, D).half()),
    dict(q=_z(B, N, 2 * HQ, D)[:, :, ::2]), dict(k_tree=_z(B, HKV, N, D).transpose(1, 2)), dict(v_tree=_z(B, N - 1, HKV, D)),
    dict(k_tree=_z(B, N, HKV, D).float()), dict(anc_mask=_i(B, N, 1)), dict(anc_mask=torch.zeros(B, N, dtype=torch.int64)),
    dict(out=_z(B, N, HQ, D).half()), dict(out=_z(B, N, HQ, 2 * D)[..., :D]), dict(out=_z(B, N - 1, HQ, D)),
    dict(lse=_z(B, N, HQ)), dict(lse=_z(B, N, HQ - 1, dtype=torch.float32)), dict(status=_i(B).long()), dict(status=_i(B - 1)),
], ids=lambda kw: next(iter(kw)))
def test_the_8bit_attention_checks_every_tensor(ts, kw):  # noqa: F811
    a = _q8_args(**kw)
    assert ts.attn_params(**a).q8_device is None
    _q8_refused(ts, a)


def test_the_8bit_attention_checks_scales_workspace_and_device(ts):  # noqa: F811
    _q8_refused(ts, _q8_args(), sc=_z(NBLK, HKV, BS, dtype=torch.uint8))
    _q8_refused(ts, _q8_args(), ws=_z(2, 1 << 20, dtype=torch.uint8)[:, ::2])
    _q8_refused(ts, _q8_args())                                   # on the CPU
    p = ts.attn_params(**_q8_args())
    assert p.q8_device == -1                                      # well formed but for that
    assert ts.attn_params(**_q8_args(lse=None, status=None, pos=None)).q8_device == -1
    assert ts.attn_params(**_q8_args(anc_mask=torch.zeros(B, N, 1, dtype=torch.uint64))).q8_device == -1
