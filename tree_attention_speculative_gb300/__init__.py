"""Python binding of libtreespec (GB300 tree-attention speculative verification).

Argument marshalling only: every function below forwards torch tensors'
device pointers, sizes and the current CUDA stream to the C entry point of
the same name in ``include/treespec.h`` and raises ``TreeSpecError`` on a
non-zero status.  All work runs in the library's CUDA kernels; there is no
other implementation behind these names, and the package refuses to work if
the library has not been built (``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Sequence

import numpy as np
import torch

from ._build import LIB as LIB_PATH

__all__ = [
    "TreeSpecError", "lib", "ts_status_str", "tree_build_ancestry", "AttnParams", "attn_params",
    "tree_attn_workspace_size", "tree_attn_plan", "tree_attn_plan_order", "tree_attn_fwd",
    "tree_verify_workspace_size", "tree_verify_greedy",
    "tree_verify_greedy_noalloc", "tree_commit_accepted", "tree_verify_stochastic", "tree_build_dynamic",
    "tree_build_ancestry_forest", "tree_verify_greedy_forest", "NOALLOC_SCRATCH_BYTES",
    "RopeConfig", "tree_rope", "tree_cache_append_q8", "tree_commit_accepted_q8",
    "tree_attn_q8_workspace_size", "tree_attn_fwd_q8", "STATUS",
]

STATUS = {
    0: "TS_OK", -1: "TS_ERR_NULL", -2: "TS_ERR_SHAPE", -3: "TS_ERR_BAD_TREE", -4: "TS_ERR_UNSUPPORTED",
    -5: "TS_ERR_BAD_BLOCK", -6: "TS_ERR_TIMEOUT", -7: "TS_ERR_CUDA", -8: "TS_ERR_WORKSPACE",
}


class TreeSpecError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({ts_status_str(status)})")


class AttnParams(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("prefix_len", ctypes.c_void_p),
        ("prefix_len_host", ctypes.c_void_p), ("k_tree", ctypes.c_void_p), ("v_tree", ctypes.c_void_p),
        ("anc_mask", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("lse", ctypes.c_void_p), ("status", ctypes.c_void_p),
        ("B", ctypes.c_int), ("N", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
        ("D", ctypes.c_int), ("block_size", ctypes.c_int), ("num_blocks", ctypes.c_int),
        ("max_blocks", ctypes.c_int), ("scale", ctypes.c_float), ("rope_theta", ctypes.c_float),
    ]


class RopeParams(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p),
        ("pos", ctypes.c_void_p),
        ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
        ("k_token_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
        ("B", ctypes.c_int), ("N", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
        ("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("scaling", ctypes.c_int),
        ("theta", ctypes.c_double), ("factor", ctypes.c_double), ("low_rot", ctypes.c_double),
        ("high_rot", ctypes.c_double), ("orig_len", ctypes.c_int), ("mscale", ctypes.c_float),
    ]


ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "bands": 3}


@dataclass(frozen=True)
class RopeConfig:
    """Rotary positions of a model (treespec.h: tree_rope).

    ``rotary_dim`` 0 rotates the whole head; ``interleaved`` pairs channels
    (2i, 2i+1) instead of (i, i + rotary_dim/2).  ``scaling``: "none",
    "linear" (positions / factor), "ntk" (base scaled by factor) or "bands"
    (frequencies that turn at least ``high_rot`` times within ``orig_len``
    tokens kept, those below ``low_rot`` divided by factor, a ramp between).
    """
    theta: float = 10000.0
    rotary_dim: int = 0
    interleaved: bool = False
    scaling: str = "none"
    factor: float = 1.0
    low_rot: float = 1.0
    high_rot: float = 4.0
    orig_len: int = 0
    mscale: float = 1.0


_LIB: Optional[ctypes.CDLL] = None

# every symbol include/treespec.h declares
EXPORTS = ("ts_status_str", "tree_build_ancestry", "tree_attn_workspace_size", "tree_attn_plan", "tree_attn_plan_order",
           "tree_attn_fwd",
           "tree_verify_workspace_size", "tree_verify_greedy", "tree_verify_greedy_noalloc",
           "tree_commit_accepted", "tree_verify_stochastic", "tree_build_dynamic", "tree_build_ancestry_forest",
           "tree_verify_greedy_forest", "tree_attn_fwd_stall_test", "tree_attn_fwd_ctas_test", "tree_rope",
           "tree_cache_append_q8", "tree_commit_accepted_q8", "tree_attn_q8_workspace_size", "tree_attn_fwd_q8",
           "tree_attn_fwd_q8_stall_test")

# TS_VERIFY_NOALLOC_SCRATCH_BYTES of treespec.h
NOALLOC_SCRATCH_BYTES = 4 << 20


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libtreespec is not built ({LIB_PATH} missing); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.ts_status_str.argtypes = [i32]
        L.ts_status_str.restype = ctypes.c_char_p
        L.tree_build_ancestry.argtypes = [vp, vp, i32, i32, vp, vp, vp, vp, vp]
        L.tree_build_ancestry.restype = i32
        L.tree_attn_workspace_size.argtypes = [ctypes.POINTER(AttnParams)]
        L.tree_attn_workspace_size.restype = sz
        L.tree_attn_plan.argtypes = [ctypes.POINTER(AttnParams), vp, vp, vp]
        L.tree_attn_plan.restype = i32
        L.tree_attn_plan_order.argtypes = [ctypes.POINTER(AttnParams), vp, i32, vp]
        L.tree_attn_plan_order.restype = i32
        L.tree_attn_fwd.argtypes = [ctypes.POINTER(AttnParams), vp, sz, vp]
        L.tree_attn_fwd.restype = i32
        L.tree_attn_fwd_stall_test.argtypes = [ctypes.POINTER(AttnParams), vp, sz, i32, i32, ctypes.c_uint32, vp]
        L.tree_attn_fwd_stall_test.restype = i32
        L.tree_attn_fwd_ctas_test.argtypes = [ctypes.POINTER(AttnParams), vp, sz, i32, i32, i32, ctypes.c_uint32, vp]
        L.tree_attn_fwd_ctas_test.restype = i32
        L.tree_verify_workspace_size.argtypes = [i32, i32, i32]
        L.tree_verify_workspace_size.restype = sz
        L.tree_verify_greedy.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]
        L.tree_verify_greedy.restype = i32
        L.tree_verify_greedy_noalloc.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp]
        L.tree_verify_greedy_noalloc.restype = i32
        L.tree_commit_accepted.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32,
                                           vp, vp, vp]
        L.tree_commit_accepted.restype = i32
        L.tree_verify_stochastic.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, ctypes.c_float, vp, vp, vp, vp,
                                             vp]
        L.tree_verify_stochastic.restype = i32
        L.tree_build_dynamic.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp]
        L.tree_build_dynamic.restype = i32
        L.tree_build_ancestry_forest.argtypes = L.tree_build_ancestry.argtypes
        L.tree_build_ancestry_forest.restype = i32
        L.tree_verify_greedy_forest.argtypes = L.tree_verify_greedy.argtypes
        L.tree_verify_greedy_forest.restype = i32
        i64 = ctypes.c_int64
        L.tree_rope.argtypes = [ctypes.POINTER(RopeParams), vp]
        L.tree_rope.restype = i32
        L.tree_cache_append_q8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i64, i64, i32, i32, i32,
                                           vp, vp, vp]
        L.tree_cache_append_q8.restype = i32
        L.tree_commit_accepted_q8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32,
                                              i32, vp, vp, vp]
        L.tree_commit_accepted_q8.restype = i32
        L.tree_attn_q8_workspace_size.argtypes = [ctypes.POINTER(AttnParams)]
        L.tree_attn_q8_workspace_size.restype = sz
        L.tree_attn_fwd_q8.argtypes = [ctypes.POINTER(AttnParams), vp, vp, sz, vp]
        L.tree_attn_fwd_q8.restype = i32
        L.tree_attn_fwd_q8_stall_test.argtypes = [ctypes.POINTER(AttnParams), vp, vp, sz, i32, i32, ctypes.c_uint32, vp]
        L.tree_attn_fwd_q8_stall_test.restype = i32
        _LIB = L
    return _LIB


def ts_status_str(status: int) -> str:
    return lib().ts_status_str(int(status)).decode()


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _s(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(st: int, where: str):
    if st != 0:
        raise TreeSpecError(st, where)


def tree_build_ancestry(parent_idx: torch.Tensor, prefix_len: torch.Tensor, anc_mask: torch.Tensor,
                        depth: torch.Tensor, pos: torch.Tensor, status: torch.Tensor, stream=None) -> None:
    """parent_idx [B,N] i32, prefix_len [B] i32 -> anc_mask [B,N,W] u64 (int64 tensor), depth, pos [B,N] i32, status [B] i32."""
    B, N = parent_idx.shape
    _check(lib().tree_build_ancestry(_p(parent_idx), _p(prefix_len), B, N, _p(anc_mask), _p(depth), _p(pos),
                                     _p(status), _s(stream)), "tree_build_ancestry")


def tree_build_ancestry_forest(parent_idx: torch.Tensor, prefix_len: torch.Tensor, anc_mask: torch.Tensor,
                               depth: torch.Tensor, pos: torch.Tensor, status: torch.Tensor, stream=None) -> None:
    """tree_build_ancestry for forests (several parent -1 entries; node 0 is a root)."""
    B, N = parent_idx.shape
    _check(lib().tree_build_ancestry_forest(_p(parent_idx), _p(prefix_len), B, N, _p(anc_mask), _p(depth), _p(pos),
                                            _p(status), _s(stream)), "tree_build_ancestry_forest")


def attn_params(q, k_cache, v_cache, block_table, prefix_len, prefix_len_host, k_tree, v_tree, anc_mask, pos,
                out, lse=None, status=None, scale: float = 0.0, rope_theta: float = 0.0) -> AttnParams:
    """Fill the C parameter block from tensors (shapes as in treespec.h).

    ``prefix_len_host`` is a host int32 tensor/array; the returned object keeps
    it alive.
    """
    B, N, Hq, D = q.shape
    nblk, Hkv, bs, _ = k_cache.shape
    host = np.ascontiguousarray(np.asarray(prefix_len_host.cpu() if torch.is_tensor(prefix_len_host)
                                           else prefix_len_host, dtype=np.int32))
    p = AttnParams(q=q.data_ptr(), k_cache=k_cache.data_ptr(), v_cache=v_cache.data_ptr(),
                   block_table=block_table.data_ptr(), prefix_len=prefix_len.data_ptr(),
                   prefix_len_host=host.ctypes.data, k_tree=k_tree.data_ptr(), v_tree=v_tree.data_ptr(),
                   anc_mask=anc_mask.data_ptr(), pos=pos.data_ptr() if pos is not None else None,
                   out=out.data_ptr(), lse=lse.data_ptr() if lse is not None else None,
                   status=status.data_ptr() if status is not None else None,
                   B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, block_size=bs, num_blocks=nblk,
                   max_blocks=block_table.shape[1], scale=scale, rope_theta=rope_theta)
    p._keep = (host,)
    p.cache_dtypes = (getattr(k_cache, "dtype", None), getattr(v_cache, "dtype", None))
    return p


def tree_attn_workspace_size(params: AttnParams) -> int:
    return int(lib().tree_attn_workspace_size(ctypes.byref(params)))


def tree_attn_plan(params: AttnParams) -> dict:
    """The split plan tree_attn_fwd uses for these arguments (host only)."""
    c, s, t = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(lib().tree_attn_plan(ctypes.byref(params), ctypes.byref(c), ctypes.byref(s), ctypes.byref(t)),
           "tree_attn_plan")
    return {"chunk_tiles": c.value, "max_splits": s.value, "tree_split": t.value}


def tree_attn_plan_order(params: AttnParams) -> list:
    """The packed (sequence, split, first tile) entries in the order the
    attention kernel takes its items (host only); [] when it orders none."""
    n = ctypes.c_int32()
    buf = (ctypes.c_uint32 * 256)()  # the most pairs the kernel orders
    _check(lib().tree_attn_plan_order(ctypes.byref(params), buf, 256, ctypes.byref(n)), "tree_attn_plan_order")
    return [int(buf[i]) for i in range(n.value)]


def tree_attn_fwd(params: AttnParams, workspace: torch.Tensor, stream=None) -> None:
    _check(lib().tree_attn_fwd(ctypes.byref(params), _p(workspace), workspace.numel() * workspace.element_size(),
                               _s(stream)), "tree_attn_fwd")


def tree_attn_fwd_stall_test(params: AttnParams, workspace: torch.Tensor, stall_seq: int, stall_tile: int,
                             wait_limit_us: int, stream=None) -> None:
    """Testing only: tree_attn_fwd with sequence ``stall_seq``'s key stream
    stopped before tile ``stall_tile``, so its bounded wait runs out."""
    _check(lib().tree_attn_fwd_stall_test(ctypes.byref(params), _p(workspace),
                                          workspace.numel() * workspace.element_size(), stall_seq, stall_tile,
                                          wait_limit_us, _s(stream)), "tree_attn_fwd_stall_test")


def tree_attn_fwd_ctas_test(params: AttnParams, workspace: torch.Tensor, max_ctas: int, stall_seq: int = -1,
                            stall_tile: int = 0, wait_limit_us: int = 1000000, stream=None) -> None:
    """Testing only: tree_attn_fwd on at most ``max_ctas`` CTAs (and, with
    ``stall_seq >= 0``, that sequence's key stream stopped as in
    tree_attn_fwd_stall_test)."""
    _check(lib().tree_attn_fwd_ctas_test(ctypes.byref(params), _p(workspace),
                                         workspace.numel() * workspace.element_size(), max_ctas, stall_seq,
                                         stall_tile, wait_limit_us, _s(stream)), "tree_attn_fwd_ctas_test")


def tree_verify_workspace_size(B: int, N: int, V: int) -> int:
    return int(lib().tree_verify_workspace_size(B, N, V))


def tree_verify_greedy(draft_tokens, target_logits, parent_idx, max_depth: int, accepted, accept_len, bonus,
                       argmax_out, status, workspace, stream=None) -> None:
    B, N, V = target_logits.shape
    _check(lib().tree_verify_greedy(_p(draft_tokens), _p(target_logits), _p(parent_idx), B, N, V, max_depth,
                                    _p(accepted), _p(accept_len), _p(bonus), _p(argmax_out), _p(status),
                                    _p(workspace), workspace.numel() * workspace.element_size(), _s(stream)),
           "tree_verify_greedy")


def tree_verify_greedy_forest(draft_tokens, target_logits, parent_idx, max_depth: int, accepted, accept_len, bonus,
                              argmax_out, status, workspace, stream=None) -> None:
    """tree_verify_greedy for forests; same workspace size."""
    B, N, V = target_logits.shape
    _check(lib().tree_verify_greedy_forest(_p(draft_tokens), _p(target_logits), _p(parent_idx), B, N, V, max_depth,
                                           _p(accepted), _p(accept_len), _p(bonus), _p(argmax_out), _p(status),
                                           _p(workspace), workspace.numel() * workspace.element_size(), _s(stream)),
           "tree_verify_greedy_forest")


def tree_commit_accepted(k_tree, v_tree, accepted, accept_len, prefix_len, k_cache, v_cache, block_table,
                         new_prefix_len, status=None, stream=None) -> None:
    """Append the accepted path (root .. n*) of every sequence to the paged cache."""
    B, N, Hkv, D = k_tree.shape
    nblk, _, bs, _ = k_cache.shape
    _check(lib().tree_commit_accepted(_p(k_tree), _p(v_tree), _p(accepted), _p(accept_len), _p(prefix_len),
                                      _p(k_cache), _p(v_cache), _p(block_table), B, N, Hkv, D, bs, nblk,
                                      block_table.shape[1], accepted.shape[1] - 1, _p(new_prefix_len), _p(status),
                                      _s(stream)), "tree_commit_accepted")


def tree_verify_stochastic(draft_tokens, target_logits, draft_probs, parent_idx, coins, temperature: float,
                           accepted, accept_len, bonus, status, stream=None) -> None:
    """Rejection-sampling verification at the given temperature; max_depth is
    accepted.shape[1] - 1.  coins [B, N] are the uniforms the walk consumes."""
    B, N, V = target_logits.shape
    _check(lib().tree_verify_stochastic(_p(draft_tokens), _p(target_logits), _p(draft_probs), _p(parent_idx),
                                        _p(coins), B, N, V, accepted.shape[1] - 1, float(temperature),
                                        _p(accepted), _p(accept_len), _p(bonus), _p(status), _s(stream)),
           "tree_verify_stochastic")


def tree_build_dynamic(pool_parent, pool_logp, pool_token, prefix_len, parent_idx, draft_tokens, sel_index,
                       anc_mask, depth, pos, status, stream=None) -> None:
    """Rerank a candidate pool [B, M] into the N-node tree of parent_idx [B, N]
    and build its masks, depths and positions."""
    B, M = pool_parent.shape
    N = parent_idx.shape[1]
    _check(lib().tree_build_dynamic(_p(pool_parent), _p(pool_logp), _p(pool_token), _p(prefix_len), B, M, N,
                                    _p(parent_idx), _p(draft_tokens), _p(sel_index), _p(anc_mask), _p(depth),
                                    _p(pos), _p(status), _s(stream)), "tree_build_dynamic")


def tree_verify_greedy_noalloc(draft_tokens, target_logits, parent_idx, max_depth: int, accepted, accept_len, bonus,
                               argmax_out, status, stream=None) -> None:
    """tree_verify_greedy without a workspace, for callers that may not allocate
    device memory (e.g. a plugin handed only its input/output buffers).  Runs on
    a fixed 4 MiB scratch array inside the library; larger problems raise
    TS_ERR_WORKSPACE.  Calls on one device share that array, so keep them
    ordered on one stream; make the first call on a device outside any stream
    capture (it looks up the array's device address)."""
    B, N, V = target_logits.shape
    _check(lib().tree_verify_greedy_noalloc(_p(draft_tokens), _p(target_logits), _p(parent_idx), B, N, V, max_depth,
                                            _p(accepted), _p(accept_len), _p(bonus), _p(argmax_out), _p(status),
                                            _s(stream)), "tree_verify_greedy_noalloc")


# ---------------------------------------------------------------- rotary positions, 8-bit cache
#
# These calls read tensors whose type and strides the C side cannot see (a bf16
# pool given as the 8-bit one would be read past its rows), so each tensor's
# type, shape, density and device are checked here first.

_CODES = (torch.float8_e4m3fn, torch.uint8)


def _need(ok: bool, where: str):
    if not ok:
        raise TreeSpecError(-2, where)  # TS_ERR_SHAPE


def _dense(where: str, t: torch.Tensor, shape, *dtypes):
    _need(t.dtype in dtypes and tuple(t.shape) == tuple(shape) and t.is_contiguous(), where)


def _same_device(where: str, *tensors):
    """Every tensor on the current CUDA device, whose stream the call uses."""
    _need(all(t is None or t.is_cuda for t in tensors), where)
    here = torch.cuda.current_device()
    _need(all(t is None or t.get_device() == here for t in tensors), where)


def _token_heads(where: str, x: torch.Tensor, out: torch.Tensor, B: int, N: int):
    """Strides (token, head) of bf16 x [B, N, H, D], whose tokens are evenly
    spaced, for the dense out of the same shape."""
    _need(x.dim() == 4 and x.dtype == torch.bfloat16 and x.shape[:2] == (B, N), where)
    _dense(where, out, x.shape, torch.bfloat16)
    sb, st, sh, sd = x.stride()
    _need((sd == 1 or x.shape[3] == 1) and (B == 1 or N == 1 or sb == N * st), where)
    H, D = x.shape[2], x.shape[3]
    if N == 1:
        st = sb if B > 1 else H * sh
    return max(st, (H - 1) * sh + D) if B * N == 1 else st, D if H == 1 else sh


def tree_rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor], pos: torch.Tensor, q_out: Optional[torch.Tensor],
              k_out: Optional[torch.Tensor], rope: RopeConfig, stream=None) -> None:
    """Rotate q [B,N,Hq,D] and k [B,N,Hkv,D] bf16 at pos [B,N] i32 into the dense
    q_out and k_out.  q and k may be views of a fused projection (evenly spaced
    tokens, adjacent channels) or the outputs themselves; either may be None."""
    B, N = pos.shape
    _dense("tree_rope", pos, (B, N), torch.int32)
    p = RopeParams(pos=pos.data_ptr(), B=B, N=N, rotary_dim=rope.rotary_dim, interleaved=int(rope.interleaved),
                   scaling=ROPE_SCALING.get(rope.scaling, -1), theta=rope.theta, factor=rope.factor,
                   low_rot=rope.low_rot, high_rot=rope.high_rot, orig_len=rope.orig_len, mscale=rope.mscale)
    if q is not None:
        _need(q_out is not None, "tree_rope")
        p.q_token_stride, p.q_head_stride = _token_heads("tree_rope", q, q_out, B, N)
        p.q, p.q_out, p.Hq, p.D = q.data_ptr(), q_out.data_ptr(), q.shape[2], q.shape[3]
    if k is not None:
        _need(k_out is not None and (q is None or k.shape[3] == q.shape[3]), "tree_rope")
        p.k_token_stride, p.k_head_stride = _token_heads("tree_rope", k, k_out, B, N)
        p.k, p.k_out, p.Hkv, p.D = k.data_ptr(), k_out.data_ptr(), k.shape[2], k.shape[3]
    _same_device("tree_rope", q, k, pos, q_out, k_out)
    _check(lib().tree_rope(ctypes.byref(p), _s(stream)), "tree_rope")


def _q8_pools(where: str, k_cache, v_cache, kv_scale, block_table, B: int, Hkv: int, D: int):
    nblk, _, bs, _ = k_cache.shape
    _dense(where, k_cache, (nblk, Hkv, bs, D), *_CODES)
    _dense(where, v_cache, (nblk, Hkv, bs, D), *_CODES)
    _dense(where, kv_scale, (nblk, Hkv, bs, 2), torch.uint8)
    _dense(where, block_table, (B, block_table.shape[1]), torch.int32)
    return nblk, bs, block_table.shape[1]


def tree_cache_append_q8(k, v, cu_len, prefix_len, k_cache, v_cache, kv_scale, block_table, new_prefix_len, status=None,
                         stream=None) -> None:
    """Quantise the new tokens k, v [T,Hkv,D] bf16 of all sequences (sequence b's
    are rows cu_len[b] .. cu_len[b+1]-1; heads dense, tokens evenly spaced) into
    the 8-bit paged cache from prefix_len on, and write new_prefix_len."""
    where = "tree_cache_append_q8"
    T, Hkv, D = k.shape
    B = prefix_len.shape[0]
    nblk, bs, maxb = _q8_pools(where, k_cache, v_cache, kv_scale, block_table, B, Hkv, D)
    for x in (k, v):
        _need(x.dtype == torch.bfloat16 and x.shape == (T, Hkv, D) and x.stride()[2] == 1
              and (Hkv == 1 or x.stride()[1] == D), where)
    _dense(where, cu_len, (B + 1,), torch.int32)
    for x in (prefix_len, new_prefix_len, status):
        if x is not None:
            _dense(where, x, (B,), torch.int32)
    _same_device(where, k, v, cu_len, prefix_len, k_cache, v_cache, kv_scale, block_table, new_prefix_len, status)
    ks, vs = (x.stride()[0] if T > 1 else 0 for x in (k, v))
    _check(lib().tree_cache_append_q8(_p(k), _p(v), _p(cu_len), _p(prefix_len), _p(k_cache), _p(v_cache),
                                      _p(kv_scale), _p(block_table), B, T, Hkv, D, ks, vs, bs, nblk, maxb,
                                      _p(new_prefix_len), _p(status), _s(stream)), where)


def tree_commit_accepted_q8(k_tree, v_tree, accepted, accept_len, prefix_len, k_cache, v_cache, kv_scale, block_table,
                            new_prefix_len, status=None, stream=None) -> None:
    """tree_commit_accepted into the 8-bit paged cache: the accepted path (root
    .. n*) of every sequence is quantised as it is appended."""
    where = "tree_commit_accepted_q8"
    B, N, Hkv, D = k_tree.shape
    nblk, bs, maxb = _q8_pools(where, k_cache, v_cache, kv_scale, block_table, B, Hkv, D)
    _dense(where, k_tree, (B, N, Hkv, D), torch.bfloat16)
    _dense(where, v_tree, (B, N, Hkv, D), torch.bfloat16)
    _dense(where, accepted, (B, accepted.shape[1]), torch.int32)
    for x in (accept_len, prefix_len, new_prefix_len, status):
        if x is not None:
            _dense(where, x, (B,), torch.int32)
    _same_device(where, k_tree, v_tree, accepted, accept_len, prefix_len, k_cache, v_cache, kv_scale, block_table,
                 new_prefix_len, status)
    _check(lib().tree_commit_accepted_q8(_p(k_tree), _p(v_tree), _p(accepted), _p(accept_len), _p(prefix_len),
                                         _p(k_cache), _p(v_cache), _p(kv_scale), _p(block_table), B, N, Hkv, D, bs,
                                         nblk, maxb, accepted.shape[1] - 1, _p(new_prefix_len), _p(status),
                                         _s(stream)), where)


def tree_attn_q8_workspace_size(params: AttnParams) -> int:
    return int(lib().tree_attn_q8_workspace_size(ctypes.byref(params)))


def _check_attn_q8(where: str, params: AttnParams, kv_scale, workspace):
    _need(all(t in _CODES for t in params.cache_dtypes), where)
    _dense(where, kv_scale, (params.num_blocks, params.Hkv, params.block_size, 2), torch.uint8)
    _same_device(where, kv_scale, workspace)


def tree_attn_fwd_q8(params: AttnParams, kv_scale: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """tree_attn_fwd over the 8-bit cache: ``params`` from attn_params with the
    e4m3 pools as k_cache and v_cache, ``kv_scale`` [num_blocks,Hkv,bs,2] uint8."""
    _check_attn_q8("tree_attn_fwd_q8", params, kv_scale, workspace)
    _check(lib().tree_attn_fwd_q8(ctypes.byref(params), _p(kv_scale), _p(workspace),
                                  workspace.numel() * workspace.element_size(), _s(stream)), "tree_attn_fwd_q8")


def tree_attn_fwd_q8_stall_test(params: AttnParams, kv_scale: torch.Tensor, workspace: torch.Tensor, stall_seq: int,
                                stall_tile: int, wait_limit_us: int, stream=None) -> None:
    """Testing only: tree_attn_fwd_q8 with sequence ``stall_seq``'s key stream
    stopped before tile ``stall_tile`` of its segments, so a bounded wait runs out."""
    where = "tree_attn_fwd_q8_stall_test"
    _check_attn_q8(where, params, kv_scale, workspace)
    _check(lib().tree_attn_fwd_q8_stall_test(ctypes.byref(params), _p(kv_scale), _p(workspace),
                                             workspace.numel() * workspace.element_size(), stall_seq, stall_tile,
                                             wait_limit_us, _s(stream)), where)
