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
    # what attn_params notes of the tensors, for the calls' checks
    cache_dtypes = ()
    q8_device = None


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
    it alive.  With 8-bit pools every tensor is checked here, for
    tree_attn_fwd_q8, which raises if one is not as treespec.h has it.
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
    p.cache_dtypes = kd, vd = getattr(k_cache, "dtype", None), getattr(v_cache, "dtype", None)
    if (kd is _F8 or kd is _U8) and (vd is _F8 or vd is _U8):
        p.q8_device = _attn_q8_device((B, N, Hq, D), (nblk, Hkv, bs, D), host, q, k_cache, v_cache, block_table,
                                      prefix_len, k_tree, v_tree, anc_mask, out, lse, status)
    return p


def _attn_q8_device(rows: tuple, pool: tuple, host, q, k_cache, v_cache, block_table, prefix_len, k_tree, v_tree,
                    anc_mask, out, lse, status):
    """The index of the device (-1: the CPU) that all of tree_attn_fwd_q8's
    tensors are on, or None if one is elsewhere or has another type, shape or
    density than the call reads."""
    B, N, Hq, D = rows
    tree = (B, N, pool[1], D)
    if not (host.shape == (B,) and _is(q, _BF16, rows) and _is(out, _BF16, rows) and _is_codes(k_cache, pool)
            and _is_codes(v_cache, pool) and _is(k_tree, _BF16, tree) and _is(v_tree, _BF16, tree)
            and _is(block_table, _I32, (B, block_table.shape[1])) and _is(prefix_len, _I32, (B,))
            and (anc_mask.dtype is torch.int64 or anc_mask.dtype is torch.uint64)
            and _is(anc_mask, anc_mask.dtype, (B, N, (N + 63) // 64))
            and (lse is None or _is(lse, torch.float32, (B, N, Hq))) and (status is None or _is(status, _I32, (B,)))):
        return None
    dev = q.get_device()
    for t in (out, k_cache, v_cache, k_tree, v_tree, block_table, prefix_len, anc_mask, lse, status):
        if t is not None and t.get_device() != dev:
            return None
    return dev


def _bf16_pools(where: str, *dtypes):
    """The bf16 calls read pools, and commit writes one, at two bytes an element:
    8-bit pools would be passed by half."""
    for d in dtypes:
        if d is not None and d.itemsize != 2:
            _bad(where)


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
    _bf16_pools("tree_attn_fwd", *params.cache_dtypes)
    _check(lib().tree_attn_fwd(ctypes.byref(params), _p(workspace), workspace.numel() * workspace.element_size(),
                               _s(stream)), "tree_attn_fwd")


def tree_attn_fwd_stall_test(params: AttnParams, workspace: torch.Tensor, stall_seq: int, stall_tile: int,
                             wait_limit_us: int, stream=None) -> None:
    """Testing only: tree_attn_fwd with sequence ``stall_seq``'s key stream
    stopped before tile ``stall_tile``, so its bounded wait runs out."""
    _bf16_pools("tree_attn_fwd_stall_test", *params.cache_dtypes)
    _check(lib().tree_attn_fwd_stall_test(ctypes.byref(params), _p(workspace),
                                          workspace.numel() * workspace.element_size(), stall_seq, stall_tile,
                                          wait_limit_us, _s(stream)), "tree_attn_fwd_stall_test")


def tree_attn_fwd_ctas_test(params: AttnParams, workspace: torch.Tensor, max_ctas: int, stall_seq: int = -1,
                            stall_tile: int = 0, wait_limit_us: int = 1000000, stream=None) -> None:
    """Testing only: tree_attn_fwd on at most ``max_ctas`` CTAs (and, with
    ``stall_seq >= 0``, that sequence's key stream stopped as in
    tree_attn_fwd_stall_test)."""
    _bf16_pools("tree_attn_fwd_ctas_test", *params.cache_dtypes)
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
    _bf16_pools("tree_commit_accepted", getattr(k_cache, "dtype", None), getattr(v_cache, "dtype", None))
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
# type, shape, density and device are checked here first.  A small call's time
# is this marshalling, so pointers go over as plain integers and the current
# stream is asked for by its handle.

_BF16, _I32, _U8, _F8 = torch.bfloat16, torch.int32, torch.uint8, torch.float8_e4m3fn


def _bad(where: str):
    raise TreeSpecError(-2, where)  # TS_ERR_SHAPE


def _is(t: torch.Tensor, dtype, shape: tuple) -> bool:
    return t.dtype is dtype and t.shape == shape and t.is_contiguous()


def _is_codes(t: torch.Tensor, shape: tuple) -> bool:
    return (t.dtype is _F8 or t.dtype is _U8) and t.shape == shape and t.is_contiguous()


def _launch_stream(where: str, stream, *tensors) -> int:
    """The stream's handle, once every tensor is on the current CUDA device."""
    for t in tensors:
        if t is not None and not t.is_cuda:
            _bad(where)
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            _bad(where)
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _opt(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _token_heads(where: str, x: torch.Tensor, out: torch.Tensor, B: int, N: int):
    """Strides (token, head) of bf16 x [B, N, H, D], whose tokens are evenly
    spaced, for the dense out of the same shape; 0, 0 when x is dense."""
    shape = x.shape
    if x.dtype is not _BF16 or len(shape) != 4 or shape[0] != B or shape[1] != N or out is None \
            or not _is(out, _BF16, shape):
        _bad(where)
    if x.is_contiguous():
        return 0, 0
    sb, st, sh, sd = x.stride()
    H, D = shape[2], shape[3]
    head = D if H == 1 else sh
    row = (H - 1) * head + D
    token = row if B * N == 1 else sb if N == 1 else st
    # (an expanded tensor repeats a token or a head: its stride of 0 would mean dense)
    if sd != 1 or not (B == 1 or N == 1 or sb == N * st) or head < D or token < row:
        _bad(where)
    return token, head


def tree_rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor], pos: torch.Tensor, q_out: Optional[torch.Tensor],
              k_out: Optional[torch.Tensor], rope: RopeConfig, stream=None) -> None:
    """Rotate q [B,N,Hq,D] and k [B,N,Hkv,D] bf16 at pos [B,N] i32 into the dense
    q_out and k_out.  q and k may be views of a fused projection (evenly spaced
    tokens, adjacent channels) or the outputs themselves; either may be None."""
    where = "tree_rope"
    B, N = pos.shape
    if pos.dtype is not _I32 or not pos.is_contiguous():
        _bad(where)
    qt = qh = kt = kh = Hq = Hkv = D = 0
    if q is not None:
        qt, qh = _token_heads(where, q, q_out, B, N)
        Hq, D = q.shape[2], q.shape[3]
    if k is not None:
        kt, kh = _token_heads(where, k, k_out, B, N)
        Hkv = k.shape[2]
        if q is not None and k.shape[3] != D:
            _bad(where)
        D = k.shape[3]
    handle = _launch_stream(where, stream, q, k, pos, q_out, k_out)
    p = RopeParams(_opt(q), _opt(k), _opt(q_out), _opt(k_out), pos.data_ptr(), qt, qh, kt, kh, B, N, Hq, Hkv, D,
                   rope.rotary_dim, rope.interleaved, ROPE_SCALING.get(rope.scaling, -1), rope.theta, rope.factor,
                   rope.low_rot, rope.high_rot, rope.orig_len, rope.mscale)
    _check(lib().tree_rope(ctypes.byref(p), handle), where)


def tree_cache_append_q8(k, v, cu_len, prefix_len, k_cache, v_cache, kv_scale, block_table, new_prefix_len, status=None,
                         stream=None) -> None:
    """Quantise the new tokens k, v [T,Hkv,D] bf16 of all sequences (sequence b's
    are rows cu_len[b] .. cu_len[b+1]-1; heads dense, tokens evenly spaced) into
    the 8-bit paged cache from prefix_len on, and write new_prefix_len."""
    where = "tree_cache_append_q8"
    T, Hkv, D = k.shape
    B = prefix_len.shape[0]
    nblk, bs, maxb = k_cache.shape[0], k_cache.shape[2], block_table.shape[1]
    pool = (nblk, Hkv, bs, D)
    ks, vs = k.stride(), v.stride()
    if not (k.dtype is _BF16 and v.dtype is _BF16 and v.shape == k.shape and ks[2] == 1 and vs[2] == 1
            and (Hkv == 1 or (ks[1] == D and vs[1] == D))
            and (T <= 1 or (ks[0] >= Hkv * D and vs[0] >= Hkv * D))
            and _is_codes(k_cache, pool) and _is_codes(v_cache, pool) and _is(kv_scale, _U8, (nblk, Hkv, bs, 2))
            and _is(block_table, _I32, (B, maxb)) and _is(cu_len, _I32, (B + 1,)) and _is(prefix_len, _I32, (B,))
            and _is(new_prefix_len, _I32, (B,)) and (status is None or _is(status, _I32, (B,)))):
        _bad(where)
    handle = _launch_stream(where, stream, k, v, cu_len, prefix_len, k_cache, v_cache, kv_scale, block_table,
                            new_prefix_len, status)
    _check(lib().tree_cache_append_q8(k.data_ptr(), v.data_ptr(), cu_len.data_ptr(), prefix_len.data_ptr(),
                                      k_cache.data_ptr(), v_cache.data_ptr(), kv_scale.data_ptr(),
                                      block_table.data_ptr(), B, T, Hkv, D, ks[0] if T > 1 else 0,
                                      vs[0] if T > 1 else 0, bs, nblk, maxb, new_prefix_len.data_ptr(), _opt(status),
                                      handle), where)


def tree_commit_accepted_q8(k_tree, v_tree, accepted, accept_len, prefix_len, k_cache, v_cache, kv_scale, block_table,
                            new_prefix_len, status=None, stream=None) -> None:
    """tree_commit_accepted into the 8-bit paged cache: the accepted path (root
    .. n*) of every sequence is quantised as it is appended."""
    where = "tree_commit_accepted_q8"
    B, N, Hkv, D = k_tree.shape
    nblk, bs, maxb = k_cache.shape[0], k_cache.shape[2], block_table.shape[1]
    pool, steps = (nblk, Hkv, bs, D), accepted.shape[1]
    if not (_is(k_tree, _BF16, (B, N, Hkv, D)) and _is(v_tree, _BF16, (B, N, Hkv, D)) and _is_codes(k_cache, pool)
            and _is_codes(v_cache, pool) and _is(kv_scale, _U8, (nblk, Hkv, bs, 2))
            and _is(block_table, _I32, (B, maxb)) and _is(accepted, _I32, (B, steps)) and _is(accept_len, _I32, (B,))
            and _is(prefix_len, _I32, (B,)) and _is(new_prefix_len, _I32, (B,))
            and (status is None or _is(status, _I32, (B,)))):
        _bad(where)
    handle = _launch_stream(where, stream, k_tree, v_tree, accepted, accept_len, prefix_len, k_cache, v_cache,
                            kv_scale, block_table, new_prefix_len, status)
    _check(lib().tree_commit_accepted_q8(k_tree.data_ptr(), v_tree.data_ptr(), accepted.data_ptr(),
                                         accept_len.data_ptr(), prefix_len.data_ptr(), k_cache.data_ptr(),
                                         v_cache.data_ptr(), kv_scale.data_ptr(), block_table.data_ptr(), B, N, Hkv,
                                         D, bs, nblk, maxb, steps - 1, new_prefix_len.data_ptr(), _opt(status),
                                         handle), where)


def tree_attn_q8_workspace_size(params: AttnParams) -> int:
    return int(lib().tree_attn_q8_workspace_size(ctypes.byref(params)))


def _attn_q8_stream(where: str, params: AttnParams, kv_scale, workspace, stream) -> int:
    if params.q8_device is None or not workspace.is_contiguous() \
            or not _is(kv_scale, _U8, (params.num_blocks, params.Hkv, params.block_size, 2)):
        _bad(where)
    handle = _launch_stream(where, stream, kv_scale, workspace)
    if params.q8_device != kv_scale.get_device():
        _bad(where)
    return handle


def tree_attn_fwd_q8(params: AttnParams, kv_scale: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """tree_attn_fwd over the 8-bit cache: ``params`` from attn_params with the
    e4m3 pools as k_cache and v_cache, ``kv_scale`` [num_blocks,Hkv,bs,2] uint8."""
    where = "tree_attn_fwd_q8"
    handle = _attn_q8_stream(where, params, kv_scale, workspace, stream)
    _check(lib().tree_attn_fwd_q8(ctypes.byref(params), kv_scale.data_ptr(), workspace.data_ptr(),
                                  workspace.numel() * workspace.element_size(), handle), where)


def tree_attn_fwd_q8_stall_test(params: AttnParams, kv_scale: torch.Tensor, workspace: torch.Tensor, stall_seq: int,
                                stall_tile: int, wait_limit_us: int, stream=None) -> None:
    """Testing only: tree_attn_fwd_q8 with sequence ``stall_seq``'s key stream
    stopped before tile ``stall_tile`` of its segments, so a bounded wait runs out."""
    where = "tree_attn_fwd_q8_stall_test"
    handle = _attn_q8_stream(where, params, kv_scale, workspace, stream)
    _check(lib().tree_attn_fwd_q8_stall_test(ctypes.byref(params), kv_scale.data_ptr(), workspace.data_ptr(),
                                             workspace.numel() * workspace.element_size(), stall_seq, stall_tile,
                                             wait_limit_us, handle), where)
