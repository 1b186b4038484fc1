"""The prompt path's calls refuse bad arguments before anything is launched (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

from tests.test_abi_host import ts  # noqa: F401
from tests.test_pool_types_host import _attn_args

NULL, SHAPE, UNSUPPORTED, WORKSPACE = -1, -2, -4, -8
B, T, HQ, HKV, D, BS, NBLK, MAXB = 3, 20, 4, 2, 64, 16, 9, 5
CU, KV = np.array([0, 7, 7, 18], np.int32), np.array([40, 3, 11], np.int32)


def _z(*s, dtype=torch.bfloat16):
    return torch.zeros(*s, dtype=dtype)


def _i(*s):
    return torch.zeros(*s, dtype=torch.int32)


def _code(ts, call):  # noqa: F811
    with pytest.raises(ts.TreeSpecError) as e:
        call()
    return e.value.status


# ------------------------------------------------------------------------------------------------- chunk attention

def _chunk(ts, **kw):  # noqa: F811
    a = dict(q=_z(T, HQ, D), k_cache=_z(NBLK, HKV, BS, D), v_cache=_z(NBLK, HKV, BS, D), block_table=_i(B, MAXB),
             cu_len=_i(B + 1), kv_len=_i(B), cu_len_host=CU, kv_len_host=KV, out=_z(T, HQ, D),
             lse=_z(T, HQ, dtype=torch.float32), status=_i(B))
    a.update(kw)
    return ts.chunk_params(**a)


def _fwd(ts, p, ws=1 << 24):  # noqa: F811
    """The C call itself (the binding would want CUDA tensors first)."""
    return ts.lib().tree_chunk_attn_fwd(ctypes.byref(p), ctypes.c_void_p(1 << 20), ws, None)


@pytest.mark.parametrize("kw", [
    dict(q=_z(T, HQ, D, dtype=torch.float16)), dict(out=_z(T, HQ, D, dtype=torch.float32)), dict(out=_z(T + 1, HQ, D)),
    dict(k_cache=_z(NBLK, HKV, BS, D, dtype=torch.uint8)), dict(v_cache=_z(NBLK, HKV, BS, D).to(torch.float8_e4m3fn)),
    dict(v_cache=_z(NBLK, HKV, BS, 2 * D)[..., ::2]), dict(q=_z(T, 2 * HQ, D)[:, ::2]), dict(cu_len=_i(B)),
    dict(kv_len=torch.zeros(B, dtype=torch.int64)), dict(cu_len_host=CU[:-1]), dict(kv_len_host=KV[:2]),
    dict(lse=_z(T, HQ)), dict(status=_i(B + 1)), dict(block_table=torch.zeros(B, MAXB, dtype=torch.int64)),
])
def test_chunk_params_refuses_tensors(ts, kw):  # noqa: F811
    assert _code(ts, lambda: _chunk(ts, **kw)) == SHAPE


@pytest.mark.parametrize("change,code", [
    (dict(q=None), NULL), (dict(cu_len=None), NULL), (dict(kv_len_host=None), NULL), (dict(block_table=None), NULL),
    (dict(D=96), UNSUPPORTED), (dict(Hq=3), SHAPE), (dict(Hq=6), UNSUPPORTED), (dict(Hq=0), SHAPE), (dict(B=0), SHAPE),
    (dict(Hq=8192, Hkv=512), UNSUPPORTED), (dict(block_size=24), UNSUPPORTED), (dict(scale=-1.0), SHAPE),
    (dict(scale=float("inf")), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(window=-1), SHAPE), (dict(sinks=-1), SHAPE),
    (dict(window=(1 << 30) + 1), UNSUPPORTED), (dict(T=17), SHAPE), (dict(max_blocks=2), SHAPE), (dict(num_blocks=0), SHAPE),
])
def test_chunk_refuses_before_launch(ts, change, code):  # noqa: F811
    p = _chunk(ts)
    assert ts.tree_chunk_attn_workspace_size(p) >= 256
    for k, v in change.items():
        setattr(p, k, v)
    assert _fwd(ts, p) == code
    assert ts.tree_chunk_attn_workspace_size(p) == 0


@pytest.mark.parametrize("cu,kv,code", [
    ([0, 7, 6, 18], KV, SHAPE), ([-1, 7, 7, 18], KV, SHAPE), ([0, 7, 7, 21], [40, 3, 30], SHAPE), (CU, [6, 3, 11], SHAPE),
    (CU, [40, -1, 11], SHAPE), (CU, [40, 3, (1 << 30) + 1], UNSUPPORTED), (CU, [40, 3, 81], SHAPE),
])
def test_chunk_refuses_lengths(ts, cu, kv, code):  # noqa: F811
    assert _fwd(ts, _chunk(ts, cu_len_host=np.array(cu, np.int32), kv_len_host=np.array(kv, np.int32))) == code


def test_chunk_refuses_alignment_and_workspaces(ts):  # noqa: F811
    p = _chunk(ts)
    need = ts.tree_chunk_attn_workspace_size(p)
    L = ts.lib()
    assert L.tree_chunk_attn_fwd(None, None, 0, None) == NULL
    assert L.tree_chunk_attn_fwd(ctypes.byref(p), None, need, None) == WORKSPACE
    assert L.tree_chunk_attn_fwd(ctypes.byref(p), ctypes.c_void_p(1 << 20), need - 1, None) == WORKSPACE
    assert L.tree_chunk_attn_fwd(ctypes.byref(p), ctypes.c_void_p((1 << 20) + 16), need, None) == WORKSPACE
    for name in ("q", "out", "k_cache", "v_cache"):
        p = _chunk(ts)
        setattr(p, name, getattr(p, name) + 8)
        assert _fwd(ts, p) == SHAPE
    assert _code(ts, lambda: ts.tree_chunk_attn_fwd(_chunk(ts), _z(need, dtype=torch.uint8), 0)) == SHAPE  # not on a GPU
    for args in ((0, -1, 0, 1000), (1, -1, 0, 99), (1, B, 0, 1000), (1, 0, -1, 1000)):
        assert L.tree_chunk_attn_fwd_test(ctypes.byref(_chunk(ts)), ctypes.c_void_p(1 << 20), need, *args, None) < 0


def test_chunk_workspace_holds_the_parts_of_cut_chains(ts):  # noqa: F811
    """One token over 60K keys of one head: 469 tiles on at most 152 SMs, each part 64 fp32 sums and a normaliser a head."""
    p = _chunk(ts, q=_z(1, 2, D), out=_z(1, 2, D), lse=None, k_cache=_z(4000, 1, BS, D), v_cache=_z(4000, 1, BS, D),
               block_table=_i(1, 4000), cu_len=_i(2), kv_len=_i(1), cu_len_host=np.array([0, 1]),
               kv_len_host=np.array([60000]), status=None)
    parts = (ts.tree_chunk_attn_workspace_size(p) - 256) / (2 * (4 * D + 4))
    assert parts == int(parts) and 16 <= parts <= 152
    # many long rows: nothing is cut
    p = _chunk(ts, q=_z(4096, 32, D), out=_z(4096, 32, D), lse=None, block_table=_i(1, 300), cu_len=_i(2), kv_len=_i(1),
               cu_len_host=np.array([0, 4096]), kv_len_host=np.array([4096]), status=None)
    assert ts.tree_chunk_attn_workspace_size(p) == 256


def test_a_few_long_chains_are_cut_beside_a_prompt(ts):  # noqa: F811
    """A prompt's 1024 tokens (32 row tiles of 24 key tiles, 8 heads) keep the SMs busy for about 50 tiles' time; the
    64-tile chains of two single tokens would outlast them, so they are cut, and nothing else is."""
    lens, past = [1024, 1, 1, 37, 1, 200, 1, 1], [2048, 8191, 4000, 0, 777, 6001, 7800, 5]
    cu = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
    T = int(cu[-1])
    p = _chunk(ts, q=_z(T, 32, 128), out=_z(T, 32, 128), lse=None, status=None, k_cache=_z(40, 8, 16, 128), v_cache=_z(40, 8, 16, 128),
               block_table=_i(8, 600), cu_len=_i(9), kv_len=_i(8), cu_len_host=cu,
               kv_len_host=np.add(lens, past).astype(np.int32))
    parts = (ts.tree_chunk_attn_workspace_size(p) - 256) / (32 * (4 * 128 + 4))
    assert parts in (4, 5, 6)  # two chains (one row each) in two or three


# ------------------------------------------------------------------------------------------------- windowed trees

@pytest.mark.parametrize("window,sinks,code", [(0, 0, SHAPE), (-3, 0, SHAPE), (4, -1, SHAPE), ((1 << 30) + 1, 0, UNSUPPORTED),
                                               (1, (1 << 30) + 1, UNSUPPORTED)])
def test_window_refuses(ts, window, sinks, code):  # noqa: F811
    p = ts.attn_params(**_attn_args())
    assert ts.tree_attn_window_workspace_size(p, 4, 1) >= 256
    assert ts.tree_attn_window_workspace_size(p, window, sinks) == 0
    L = ts.lib()
    assert L.tree_attn_fwd_window(ctypes.byref(p), window, sinks, ctypes.c_void_p(1 << 20), 1 << 24, None) == code
    assert L.tree_attn_fwd_window(ctypes.byref(p), 4, 1, None, 1 << 24, None) == WORKSPACE
    p.D = 96
    assert L.tree_attn_fwd_window(ctypes.byref(p), 4, 1, ctypes.c_void_p(1 << 20), 1 << 24, None) == UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(k_cache=torch.zeros(9, 2, 16, 64, dtype=torch.uint8)), dict(q=torch.zeros(3, 6, 4, 64)),
    dict(anc_mask=torch.zeros(3, 6, 2, dtype=torch.int64)), dict(k_tree=torch.zeros(3, 6, 1, 64, dtype=torch.bfloat16)),
    dict(prefix_len=torch.zeros(3, dtype=torch.int64)), dict(prefix_len_host=np.zeros(2, np.int32)), dict(),
])
def test_window_refuses_tensors(ts, kw):  # noqa: F811
    """Wrong types and shapes, and (the last) tensors that are not on a GPU."""
    p = ts.attn_params(**_attn_args(**kw))
    assert _code(ts, lambda: ts.tree_attn_fwd_window(p, 4, 1, _z(1 << 20, dtype=torch.uint8), 0)) == SHAPE


# ------------------------------------------------------------------------------------------------- rotated appends

def _append(ts, rope="plain", **kw):  # noqa: F811
    a = dict(q=_z(T, HQ, D), k=_z(T, HKV, D), v=_z(T, HKV, D), cu_len=_i(B + 1), prefix_len=_i(B), q_out=_z(T, HQ, D),
             k_cache=_z(NBLK, HKV, BS, D), v_cache=_z(NBLK, HKV, BS, D), block_table=_i(B, MAXB), new_prefix_len=_i(B),
             rope=ts.RopeConfig() if rope == "plain" else rope, status=_i(B))
    a.update(kw)
    return lambda: ts.tree_cache_append_rope(**a, stream=0)


U8 = dict(dtype=torch.uint8)


@pytest.mark.parametrize("kw", [
    dict(), dict(q=_z(T, HQ, D, dtype=torch.float32)), dict(q_out=None), dict(q_out=_z(T, HQ, 2 * D)[..., ::2]),
    dict(k=_z(T, 2 * HKV, D)[:, :, ::1][:, ::2][:, :1].expand(T, HKV, D)), dict(v=_z(T, HKV, 2 * D)[..., ::2]),
    dict(v=_z(1, HKV, D).expand(T, HKV, D)), dict(k_cache=_z(NBLK, HKV, BS, D, **U8)), dict(cu_len=_i(B)),
    dict(kv_scale=_z(NBLK, HKV, BS, 2, **U8)),  # scales with bf16 pools
    dict(k_cache=_z(NBLK, HKV, BS, D, **U8), v_cache=_z(NBLK, HKV, BS, D, **U8), kv_scale=_z(NBLK, HKV, BS, **U8)),
    dict(status=_i(B + 1)), dict(new_prefix_len=_z(B, dtype=torch.float32)), dict(block_table=_i(B + 1, MAXB)),
])
def test_append_refuses_tensors(ts, kw):  # noqa: F811
    """Wrong types, shapes and strides, and (the first) tensors that are not on a GPU."""
    assert _code(ts, _append(ts, **kw)) == SHAPE


def _append_block(ts, **change):  # noqa: F811
    rope = ts.RopeParams(theta=10000.0, factor=1.0, low_rot=1.0, high_rot=4.0, mscale=1.0)
    at = iter(range(1 << 20, 1 << 30, 1 << 20))
    names = ("q", "k", "v", "q_out", "k_cache", "v_cache", "cu_len", "prefix_len", "block_table", "new_prefix_len", "status")
    p = ts.AppendParams(**{n: next(at) for n in names}, rope=ctypes.pointer(rope), B=B, T=T, Hq=HQ, Hkv=HKV, D=D,
                        block_size=BS, num_blocks=NBLK, max_blocks=MAXB)
    for k, v in change.items():
        if k.startswith("rope_"):
            setattr(rope, k[5:], v)
        elif isinstance(v, str):
            setattr(p, k, getattr(p, v))
        else:
            setattr(p, k, v)
    p._keep = rope
    return ts.lib().tree_cache_append_rope(bytes(p), None)


@pytest.mark.parametrize("change,code", [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(q_out=None), NULL), (dict(cu_len=None), NULL), (dict(k_cache=None), NULL),
    (dict(new_prefix_len=None), NULL), (dict(rope=None), NULL), (dict(B=0), SHAPE), (dict(T=-1), SHAPE), (dict(Hkv=0), SHAPE),
    (dict(Hq=0), SHAPE), (dict(D=80), UNSUPPORTED), (dict(Hq=4097), UNSUPPORTED), (dict(block_size=8), UNSUPPORTED),
    (dict(q_token_stride=HQ * D - 8), SHAPE), (dict(k_head_stride=D + 4), SHAPE), (dict(v_token_stride=4), SHAPE),
    (dict(k=(3 << 20) + 2), SHAPE), (dict(kv_scale=(64 << 20) + 1), SHAPE), (dict(q_out="q"), SHAPE), (dict(q_out="k"), SHAPE),
    (dict(new_prefix_len="prefix_len"), SHAPE), (dict(new_prefix_len="cu_len"), SHAPE), (dict(status="new_prefix_len"), SHAPE),
    (dict(rope_rotary_dim=3), SHAPE), (dict(rope_rotary_dim=D + 2), SHAPE), (dict(rope_theta=0.0), SHAPE),
    (dict(rope_mscale=float("nan")), SHAPE), (dict(rope_scaling=7), UNSUPPORTED), (dict(rope_scaling=3), SHAPE),
])
def test_append_refuses_before_launch(ts, change, code):  # noqa: F811
    assert _append_block(ts, **change) == code
    assert ts.lib().tree_cache_append_rope(None, None) == NULL


# ------------------------------------------------------------------------------------------------- log probabilities

def _logp(ts, **kw):  # noqa: F811
    f = dict(dtype=torch.float32)
    a = dict(logits=_z(6, 50, **f), tokens=_i(4), logprob=_z(4, **f), entropy=_z(4, **f), top_ids=_i(4, 3),
             top_logprobs=_z(4, 3, **f), rows=_i(4))
    a.update(kw)
    return lambda: ts.tree_token_logprobs(**a, stream=0)


@pytest.mark.parametrize("kw", [
    dict(), dict(logits=_z(6, 50, dtype=torch.float16)), dict(logits=_z(50, 6, dtype=torch.float32).t()),
    dict(logits=_z(1, 50, dtype=torch.float32).expand(6, 50)), dict(logits=_z(4, 6, 50, dtype=torch.float32)[::2, :5]),
    dict(tokens=_i(5)), dict(tokens=torch.zeros(4, dtype=torch.int64)), dict(logprob=_z(4)), dict(entropy=_z(4, dtype=torch.float64)),
    dict(top_ids=_i(4, 2)), dict(top_logprobs=_z(3, 3, dtype=torch.float32)), dict(rows=_i(3)),
    dict(logprob=None, entropy=None, top_ids=None, top_logprobs=None),
])
def test_logprobs_refuses_tensors(ts, kw):  # noqa: F811
    """Wrong types, shapes and strides, and (the first) tensors that are not on a GPU."""
    assert _code(ts, _logp(ts, **kw)) == SHAPE


@pytest.mark.parametrize("change,code", [
    (dict(logits=None), NULL), (dict(tokens=None), NULL), (dict(logprob=None), NULL), (dict(top=0), NULL),
    (dict(top_ids=None, top_logprobs=None), NULL), (dict(R=-1), SHAPE), (dict(V=0), SHAPE), (dict(top=33), UNSUPPORTED),
    (dict(V=524225, row_stride=0), UNSUPPORTED), (dict(row_stride=49), SHAPE), (dict(temperature=0.0), SHAPE),
    (dict(temperature=-1.0), SHAPE), (dict(temperature=float("inf")), SHAPE), (dict(temperature=float("nan")), SHAPE),
    (dict(temperature=1e-45), SHAPE), (dict(rows=None, M=3), SHAPE), (dict(logits=(1 << 20) + 2), SHAPE),
    (dict(logits=(1 << 20) + 1, half=1), SHAPE),
])
def test_logprobs_refuses_before_launch(ts, change, code):  # noqa: F811
    p = ts.LogprobParams(logits=1 << 20, tokens=2 << 20, rows=3 << 20, logprob=4 << 20, entropy=5 << 20, top_ids=6 << 20,
                         top_logprobs=7 << 20, row_stride=50, R=4, M=6, V=50, top=3, half=0, temperature=1.0)
    for k, v in change.items():
        setattr(p, k, v)
    assert ts.lib().tree_token_logprobs(ctypes.byref(p), None) == code


def test_a_windowed_step_refuses_the_8bit_cache(ts):  # noqa: F811
    from tree_attention_speculative_gb300.step import TreeVerifyStep
    step = TreeVerifyStep(B, 6, HQ, HKV, D, np.zeros(B, np.int32), device="cpu", window=8)
    a = _attn_args()
    with pytest.raises(ValueError):
        step.attention(a["q"], a["k_cache"], a["v_cache"], a["block_table"], a["prefix_len"], a["k_tree"], a["v_tree"], 0,
                       kv_scale=_z(NBLK, HKV, BS, 2, dtype=torch.uint8))
