"""Refusals of the rope and 8-bit cache calls, made before anything is launched (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

from tests.test_abi_host import _FakeTensor, _params, ts  # noqa: F401

A = 0x100000     # a fake aligned address; the buffers below lie 16 MB apart
NULL, SHAPE, UNSUPPORTED, WORKSPACE = -1, -2, -4, -8


def _at(i):
    return A + i * (16 << 20)


def _rope(ts, **kw):
    p = dict(q=_at(0), k=_at(1), q_out=_at(2), k_out=_at(3), pos=_at(4), B=2, N=5, Hq=8, Hkv=2, D=128, theta=10000.0,
             factor=1.0, low_rot=1.0, high_rot=4.0, mscale=1.0)
    p.update(kw)
    return ts.lib().tree_rope(ctypes.byref(ts.RopeParams(**p)), None)


@pytest.mark.parametrize("kw,want", [
    (dict(pos=None), NULL), (dict(q=None, k=None), NULL), (dict(q_out=None), NULL), (dict(k_out=None), NULL),
    (dict(B=0), SHAPE), (dict(N=0), SHAPE), (dict(Hq=0), SHAPE), (dict(Hkv=0), SHAPE), (dict(B=65536, N=65536), SHAPE),
    (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED), (dict(Hq=5000), UNSUPPORTED),
    (dict(scaling=4), UNSUPPORTED), (dict(scaling=-1), UNSUPPORTED),
    (dict(rotary_dim=3), SHAPE), (dict(rotary_dim=130), SHAPE), (dict(rotary_dim=-2), SHAPE),
    (dict(theta=0.0), SHAPE), (dict(theta=float("inf")), SHAPE), (dict(theta=float("nan")), SHAPE), (dict(mscale=0.0), SHAPE),
    (dict(scaling=1, factor=0.0), SHAPE), (dict(scaling=2, factor=float("nan")), SHAPE),
    (dict(scaling=3, factor=8.0, orig_len=0), SHAPE), (dict(scaling=3, factor=8.0, orig_len=4096, low_rot=4.0), SHAPE),
    (dict(q=_at(0) + 8), SHAPE), (dict(k_out=_at(3) + 2), SHAPE),
    (dict(q_head_stride=120), SHAPE), (dict(q_head_stride=132), SHAPE), (dict(q_token_stride=1000), SHAPE),
    (dict(k_token_stride=-256), SHAPE), (dict(k_token_stride=260), SHAPE),
    # overlaps: shifted in place; in place with strides; an output over the other input, the other output, pos
    (dict(q_out=_at(0) + 128), SHAPE), (dict(q_out=_at(0), q_token_stride=2048), SHAPE), (dict(q_out=_at(1)), SHAPE),
    (dict(k_out=_at(2) + 16), SHAPE), (dict(k_out=_at(4) - 64), SHAPE),
])
def test_rope_refuses(ts, kw, want):  # noqa: F811
    assert _rope(ts, **kw) == want


def _append(ts, **kw):
    p = dict(k=_at(0), v=_at(1), cu=_at(2), plen=_at(3), kc=_at(4), vc=_at(5), sc=_at(6), table=_at(7), B=2, T=10, Hkv=2,
             D=128, ks=0, vs=0, bs=16, nblk=9, maxb=3, new=_at(8), status=_at(9))
    p.update(kw)
    return ts.lib().tree_cache_append_q8(*p.values(), None)


@pytest.mark.parametrize("kw,want", [
    *[({name: None}, NULL) for name in ("k", "v", "cu", "plen", "kc", "vc", "sc", "table", "new")],
    (dict(B=0), SHAPE), (dict(T=-1), SHAPE), (dict(Hkv=0), SHAPE), (dict(bs=0), SHAPE), (dict(nblk=0), SHAPE),
    (dict(maxb=0), SHAPE), (dict(D=80), UNSUPPORTED), (dict(bs=24), UNSUPPORTED), (dict(Hkv=5000), UNSUPPORTED),
    (dict(ks=200), SHAPE), (dict(vs=260), SHAPE), (dict(k=_at(0) + 8), SHAPE), (dict(sc=_at(6) + 2), SHAPE),
    (dict(vc=_at(5) + 8), SHAPE), (dict(new=_at(3)), SHAPE), (dict(new=_at(3) + 4), SHAPE), (dict(new=_at(2) + 8), SHAPE),
    (dict(new=_at(9)), SHAPE),
])
def test_append_refuses(ts, kw, want):  # noqa: F811
    assert _append(ts, **kw) == want


def _commit(ts, **kw):
    p = dict(k=_at(0), v=_at(1), acc=_at(2), alen=_at(3), plen=_at(4), kc=_at(5), vc=_at(6), sc=_at(7), table=_at(8), B=2,
             N=10, Hkv=2, D=128, bs=16, nblk=9, maxb=3, depth=4, new=_at(9), status=None)
    p.update(kw)
    return ts.lib().tree_commit_accepted_q8(*p.values(), None)


@pytest.mark.parametrize("kw,want", [
    *[({name: None}, NULL) for name in ("k", "v", "acc", "alen", "plen", "kc", "vc", "sc", "table", "new")],
    (dict(B=0), SHAPE), (dict(N=257), SHAPE), (dict(Hkv=0), SHAPE), (dict(bs=0), SHAPE), (dict(depth=-1), SHAPE),
    (dict(D=32), UNSUPPORTED), (dict(bs=40), UNSUPPORTED), (dict(k=_at(0) + 4), SHAPE), (dict(sc=_at(7) + 1), SHAPE),
])
def test_commit_refuses(ts, kw, want):  # noqa: F811
    assert _commit(ts, **kw) == want


def test_attn_q8_refuses(ts):  # noqa: F811
    L = ts.lib()
    p = _params(ts)
    n = ts.tree_attn_q8_workspace_size(p)
    assert n >= 256
    call = lambda p, sc=A, ws=A, size=n: L.tree_attn_fwd_q8(ctypes.byref(p), sc, ws, size, None)  # noqa: E731
    assert call(p, sc=None) == NULL and call(p, sc=A + 8) == SHAPE
    assert call(p, ws=None) == WORKSPACE and call(p, size=n - 1) == WORKSPACE and call(p, ws=A + 16) == WORKSPACE
    for bad, want in ((dict(D=96), UNSUPPORTED), (dict(N=257), UNSUPPORTED), (dict(Hq=24, Hkv=8), UNSUPPORTED),
                      (dict(Hq=12, Hkv=8), SHAPE), (dict(bs=24), UNSUPPORTED), (dict(P=(-1, 5)), SHAPE)):
        q = _params(ts, **bad)
        assert call(q) == want and ts.tree_attn_q8_workspace_size(q) == 0
    q = _params(ts)
    q.rope_theta = 10000.0
    assert call(q) == UNSUPPORTED


def test_binding_checks_types_and_shapes(ts):  # noqa: F811
    """A wrong type, shape or density raises before any pointer is passed on."""
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    u = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    cfg = ts.RopeConfig()
    q, k, pos = z(2, 5, 8, 64), z(2, 5, 2, 64), i(2, 5)
    for bad in (dict(pos=pos.long()), dict(q=q.float()), dict(q_out=q[:, :4]), dict(k=z(2, 4, 2, 64)), dict(k_out=None),
                dict(q=z(2, 5, 8, 128)[..., ::2]), dict(q_out=z(2, 5, 16, 64)[:, :, ::2])):
        a = dict(q=q, k=k, pos=pos, q_out=q.clone(), k_out=k.clone(), rope=cfg)
        a.update(bad)
        with pytest.raises((ts.TreeSpecError, AttributeError)):
            ts.tree_rope(**a)
    a = dict(k=z(7, 2, 64), v=z(7, 2, 64), cu_len=i(4), prefix_len=i(3), k_cache=u(9, 2, 16, 64), v_cache=u(9, 2, 16, 64),
             kv_scale=u(9, 2, 16, 2), block_table=i(3, 5), new_prefix_len=i(3))
    for bad in (dict(k_cache=z(9, 2, 16, 64)), dict(v_cache=u(9, 2, 16, 128)), dict(kv_scale=u(9, 2, 16)), dict(cu_len=i(3)),
                dict(v=z(6, 2, 64)), dict(k=z(7, 2, 64).half()), dict(k=z(7, 64, 2).transpose(1, 2)), dict(block_table=i(2, 5)),
                dict(new_prefix_len=i(4)), dict(prefix_len=torch.zeros(3, dtype=torch.int64))):
        with pytest.raises(ts.TreeSpecError):
            ts.tree_cache_append_q8(**{**a, **bad})
    a = dict(k_tree=z(3, 6, 2, 64), v_tree=z(3, 6, 2, 64), accepted=i(3, 4), accept_len=i(3), prefix_len=i(3),
             k_cache=u(9, 2, 16, 64), v_cache=u(9, 2, 16, 64), kv_scale=u(9, 2, 16, 2), block_table=i(3, 5), new_prefix_len=i(3))
    for bad in (dict(v_tree=z(3, 6, 2, 128)), dict(accepted=i(2, 4)), dict(accept_len=i(2)), dict(k_cache=z(9, 2, 16, 64)),
                dict(kv_scale=u(9, 16, 2, 2).transpose(1, 2))):
        with pytest.raises(ts.TreeSpecError):
            ts.tree_commit_accepted_q8(**{**a, **bad})
    with pytest.raises(ts.TreeSpecError):   # bf16 pools
        p = ts.attn_params(z(3, 6, 4, 64), z(9, 2, 16, 64), z(9, 2, 16, 64), i(3, 5), i(3), np.zeros(3, np.int32),
                           z(3, 6, 2, 64), z(3, 6, 2, 64), torch.zeros(3, 6, 1, dtype=torch.int64), None, z(3, 6, 4, 64))
        ts.tree_attn_fwd_q8(p, u(9, 2, 16, 2), u(1024))


def test_stall_test_refuses(ts):  # noqa: F811
    p = _params(ts)
    n = ts.tree_attn_q8_workspace_size(p)
    call = lambda seq, tile, us: ts.lib().tree_attn_fwd_q8_stall_test(ctypes.byref(p), A, A, n, seq, tile, us, None)  # noqa: E731
    assert call(-1, 0, 1000) == SHAPE and call(2, 0, 1000) == SHAPE and call(0, -1, 1000) == SHAPE
    assert call(0, 0, 99) == UNSUPPORTED and call(0, 0, 1000001) == UNSUPPORTED
