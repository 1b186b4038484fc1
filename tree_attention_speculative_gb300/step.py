"""Steps on the GPU: device buffers plus the library's calls.

``TreeVerifyStep`` owns the output and workspace buffers (allocated with torch,
which is only the allocator here) for fixed sizes and enqueues
tree_build_ancestry -> tree_attn_fwd -> tree_verify_greedy on one stream (their
_forest variants with ``forest=True``).  With a ``rope`` configuration it
positions q and k_tree in between (tree_rope), with ``kv_scale`` it reads an
8-bit cache (tree_attn_fwd_q8), and ``commit`` appends the accepted path to
either cache.  With a ``window`` it is the step of a windowed layer
(tree_attn_fwd_window), and ``logprobs`` scores the accepted path
(tree_token_logprobs).  Every computation happens in the library's kernels (the
accepted path's rows are picked with a few of torch's index operations).

``PromptStep`` is the step that fills the cache: a ragged batch of prompts, chunks of
them or decoded tokens goes through tree_cache_append_rope, tree_chunk_attn_fwd
and, for its logits, tree_token_logprobs.

``PackedInputs`` stages a step's inputs from host memory in one copy.
"""
from __future__ import annotations

from typing import Optional

import numpy as np
import torch

from . import (RopeConfig, attn_params, chunk_params, tree_attn_fwd, tree_attn_fwd_q8, tree_attn_fwd_window,
               tree_attn_q8_workspace_size, tree_attn_window_workspace_size, tree_attn_workspace_size,
               tree_build_ancestry, tree_build_ancestry_forest, tree_cache_append_rope, tree_chunk_attn_fwd,
               tree_chunk_attn_workspace_size, tree_commit_accepted, tree_commit_accepted_q8, tree_rope,
               tree_token_logprobs, tree_verify_greedy, tree_verify_greedy_forest, tree_verify_workspace_size)


class PackedInputs:
    """A step's inputs packed into one pinned host buffer and one device buffer
    (every tensor at a 256-byte aligned offset), so that the whole host-to-device
    upload of a step is a single copy, which can run on a stream of its own
    while the previous step computes.

    ``arrays`` maps names to CPU tensors (any dtype); ``device(name)`` is the
    device view to hand to the library's calls, ``upload(stream)`` enqueues the
    copy.  Torch is only the allocator and the copy call here.
    """

    ALIGN = 256

    def __init__(self, arrays: dict, device):
        self.layout = {}
        off = 0
        for name, t in arrays.items():
            t = t.contiguous()
            self.layout[name] = (off, tuple(t.shape), t.dtype)
            off += -(-(t.numel() * t.element_size()) // self.ALIGN) * self.ALIGN
        self.nbytes = off
        self.host = torch.empty(off, dtype=torch.uint8)
        if torch.device(device).type == "cuda":
            self.host = self.host.pin_memory()
        self.dev = torch.empty(off, dtype=torch.uint8, device=device)
        for name, t in arrays.items():
            self.host_view(name).copy_(t)

    def _view(self, buf: torch.Tensor, name: str) -> torch.Tensor:
        off, shape, dtype = self.layout[name]
        n = int(np.prod(shape, dtype=np.int64)) * torch.empty((), dtype=dtype).element_size()
        return buf[off:off + n].view(dtype).view(shape)

    def host_view(self, name: str) -> torch.Tensor:
        return self._view(self.host, name)

    def device(self, name: str) -> torch.Tensor:
        return self._view(self.dev, name)

    def upload(self, stream=None) -> None:
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(self.dev.device)):
            self.dev.copy_(self.host, non_blocking=True)


def _on(stream, device):
    """Makes ``stream`` (a torch stream, a handle, or None: the current one) current, so that
    what is made for a call is filled before it."""
    if stream is None or device.type != "cuda":
        return torch.cuda.stream(None)
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device))


def _grown(step, name: str, need: int, stream=None) -> torch.Tensor:
    """The step's workspace of that name, of ``need`` bytes at least.  One that grew too
    small stays allocated: captured calls still write to it."""
    ws = getattr(step, name)
    if ws is None or ws.numel() < need:
        if ws is not None:
            step.outgrown.append(ws)
            need = max(need, 2 * ws.numel())  # so that what is kept stays below the one in use
        # zero-filled once; every call leaves its head (the item counter) zero again
        with _on(stream, step.device):
            ws = torch.zeros(need, dtype=torch.uint8, device=step.device)
        setattr(step, name, ws)
    return ws


class _Scores:
    """Outputs of tree_token_logprobs for ``rows`` rows."""

    def __init__(self, rows: int, top: int, device):
        f32 = dict(dtype=torch.float32, device=device)
        self.logprob, self.entropy = torch.zeros(rows, **f32), torch.zeros(rows, **f32)
        self.top_ids = torch.full((rows, top), -1, dtype=torch.int32, device=device) if top else None
        self.top_logprobs = torch.zeros(rows, top, **f32) if top else None


class TreeVerifyStep:
    def __init__(self, B: int, N: int, Hq: int, Hkv: int, D: int, prefix_len_host, vocab: int = 0,
                 max_depth: Optional[int] = None, device="cuda", scale: float = 0.0, forest: bool = False,
                 rope: Optional[RopeConfig] = None, window: int = 0, sinks: int = 0):
        self.B, self.N, self.Hq, self.Hkv, self.D = B, N, Hq, Hkv, D
        self.forest = forest
        self.vocab = vocab
        self.max_depth = N - 1 if max_depth is None else max_depth
        self.scale = scale
        self.window, self.sinks = window, sinks  # a window of 0: every prefix token is visible
        self.device = torch.device(device)
        self.prefix_len_host = np.ascontiguousarray(np.asarray(prefix_len_host, np.int32))
        W = (N + 63) // 64
        dev = self.device
        i32 = dict(dtype=torch.int32, device=dev)
        self.anc = torch.zeros(B, N, W, dtype=torch.int64, device=dev)
        self.depth = torch.zeros(B, N, **i32)
        self.pos = torch.zeros(B, N, **i32)
        self.status = torch.zeros(B, **i32)
        self.out = torch.empty(B, N, Hq, D, dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty(B, N, Hq, dtype=torch.float32, device=dev)
        self.ws_attn = None
        self.ws_attn_q8 = None  # of its own: a captured bf16 call keeps the other
        self.outgrown = []  # workspaces that grew too small: captured calls still write to them
        self.rope = rope
        if rope is not None:
            self.q_rot = torch.empty(B, N, Hq, D, dtype=torch.bfloat16, device=dev)
            self.k_rot = torch.empty(B, N, Hkv, D, dtype=torch.bfloat16, device=dev)
        if vocab > 0:
            nb = tree_verify_workspace_size(B, N, vocab)
            # zero-filled once; the verify kernel leaves its counters at zero
            self.ws_verify = torch.zeros(nb, dtype=torch.uint8, device=dev)
            self.accepted = torch.empty(B, self.max_depth + 1, **i32)
            self.accept_len = torch.empty(B, **i32)
            self.bonus = torch.empty(B, **i32)
            self.argmax = torch.empty(B, N, **i32)

    def _params(self, q, k_cache, v_cache, block_table, prefix_len, k_tree, v_tree):
        return attn_params(q, k_cache, v_cache, block_table, prefix_len, self.prefix_len_host, k_tree, v_tree,
                           self.anc, self.pos, self.out, self.lse, self.status, scale=self.scale)

    def _workspace_bytes(self, p, kv_scale) -> int:
        if self.window and kv_scale is not None:
            raise ValueError("a windowed layer's cache is bf16")
        if self.window:
            return tree_attn_window_workspace_size(p, self.window, self.sinks)
        return tree_attn_workspace_size(p) if kv_scale is None else tree_attn_q8_workspace_size(p)

    def attn_workspace_bytes(self, q, k_cache, v_cache, block_table, prefix_len, k_tree, v_tree, kv_scale=None) -> int:
        """The bytes that ``attention`` needs for these arguments."""
        return self._workspace_bytes(self._params(q, k_cache, v_cache, block_table, prefix_len, k_tree, v_tree), kv_scale)

    def ancestry(self, parent, prefix_len, stream=None):
        build = tree_build_ancestry_forest if self.forest else tree_build_ancestry
        build(parent, prefix_len, self.anc, self.depth, self.pos, self.status, stream)

    def position(self, q, k_tree, stream=None):
        """q and k_tree rotated at the nodes' positions (their own tensors
        without a rope configuration); the rotated keys are what commit appends."""
        if self.rope is None:
            return q, k_tree
        tree_rope(q, k_tree, self.pos, self.q_rot, self.k_rot, self.rope, stream)
        return self.q_rot, self.k_rot

    def attention(self, q, k_cache, v_cache, block_table, prefix_len, k_tree, v_tree, stream=None, kv_scale=None):
        p = self._params(q, k_cache, v_cache, block_table, prefix_len, k_tree, v_tree)
        need = self._workspace_bytes(p, kv_scale)
        if need == 0:
            raise ValueError("tree_attn_fwd would reject these arguments")
        ws = _grown(self, "ws_attn" if kv_scale is None else "ws_attn_q8", need, stream)
        if self.window:
            tree_attn_fwd_window(p, self.window, self.sinks, ws, stream)
        elif kv_scale is None:
            tree_attn_fwd(p, ws, stream)
        else:
            tree_attn_fwd_q8(p, kv_scale, ws, stream)

    def verify(self, draft, logits, parent, stream=None):
        verify = tree_verify_greedy_forest if self.forest else tree_verify_greedy
        verify(draft, logits, parent, self.max_depth, self.accepted, self.accept_len, self.bonus, self.argmax,
               self.status, self.ws_verify, stream)

    def run(self, parent, prefix_len, q, k_cache, v_cache, block_table, k_tree, v_tree, draft=None, logits=None,
            stream=None, kv_scale=None):
        self.ancestry(parent, prefix_len, stream)
        q, k_tree = self.position(q, k_tree, stream)
        self.attention(q, k_cache, v_cache, block_table, prefix_len, k_tree, v_tree, stream, kv_scale)
        if logits is not None:
            self.verify(draft, logits, parent, stream)

    def commit(self, k_tree, v_tree, prefix_len, k_cache, v_cache, block_table, new_prefix_len, stream=None,
               kv_scale=None):
        """Append the accepted path of the last ``run`` (with a rope configuration
        its rotated keys, in place of k_tree) to the bf16 cache, or to the 8-bit
        one with its ``kv_scale``."""
        k = k_tree if self.rope is None else self.k_rot
        if kv_scale is None:
            tree_commit_accepted(k, v_tree, self.accepted, self.accept_len, prefix_len, k_cache, v_cache, block_table,
                                 new_prefix_len, self.status, stream)
        else:
            tree_commit_accepted_q8(k, v_tree, self.accepted, self.accept_len, prefix_len, k_cache, v_cache, kv_scale,
                                    block_table, new_prefix_len, self.status, stream)

    def logprobs(self, draft, logits, temperature: float = 1.0, top: int = 0, stream=None) -> _Scores:
        """Log probabilities of the tokens the last ``run`` emitted: row b (max_depth + 1)
        + d scores the token after path step d, the next accepted draft or at the end
        the bonus, under that step's logits.  Rows past a path stay 0 (ids -1)."""
        with _on(stream, self.device):
            path, after = self.accepted, torch.cat((self.accepted[:, 1:], self.accepted.new_full((self.B, 1), -1)), 1)
            base = torch.arange(self.B, dtype=torch.int32, device=self.device)[:, None] * self.N
            rows = torch.where(path >= 0, base + path, -1).view(-1)
            tokens = torch.where(after >= 0, draft.gather(1, after.clamp(min=0).long()), self.bonus[:, None])
            out = _Scores(rows.numel(), top, self.device)
            tree_token_logprobs(logits, tokens.int().view(-1).contiguous(), out.logprob, out.entropy, out.top_ids,
                                out.top_logprobs, rows=rows.contiguous(), temperature=temperature)
        return out


class PromptStep:
    """One layer's pass over a ragged batch of new tokens (sequence b's are rows
    cu_len[b] .. cu_len[b+1]-1, at most ``max_tokens`` in all): ``run`` appends them to
    the paged cache with their rotary positions and attends; ``score`` gives the
    log probabilities of the tokens that followed.  ``window`` and ``sinks`` are those
    of a windowed layer (0: none).  ``status`` keeps a sequence's error: nothing more is
    appended to it, and no rows of its are attended, until the caller has set it back to 0."""

    def __init__(self, B: int, max_tokens: int, Hq: int, Hkv: int, D: int, rope: RopeConfig, device="cuda",
                 scale: float = 0.0, window: int = 0, sinks: int = 0):
        self.B, self.Hq, self.Hkv, self.D = B, Hq, Hkv, D
        self.rope, self.scale, self.window, self.sinks = rope, scale, window, sinks
        self.device = dev = torch.device(device)
        self.q_rot = torch.zeros(max_tokens, Hq, D, dtype=torch.bfloat16, device=dev)
        self.out = torch.zeros(max_tokens, Hq, D, dtype=torch.bfloat16, device=dev)
        self.lse = torch.zeros(max_tokens, Hq, dtype=torch.float32, device=dev)
        self.kv_len = torch.zeros(B, dtype=torch.int32, device=dev)
        self.status = torch.zeros(B, dtype=torch.int32, device=dev)
        self.appended = torch.full((B,), 1 << 30, dtype=torch.int32, device=dev)  # (before the first append: any rows)
        self.ws_attn = None
        self.outgrown = []

    def append(self, q, k, v, cu_len, prefix_len, k_cache, v_cache, block_table, kv_scale=None, stream=None):
        """The tokens into the cache (with ``kv_scale`` the 8-bit one); the rotated queries
        and, in ``kv_len`` and ``appended``, the sequences' new lengths and how much longer
        they have become."""
        q_rot = None if q is None else self.q_rot[:q.shape[0]]
        tree_cache_append_rope(q, k, v, cu_len, prefix_len, q_rot, k_cache, v_cache, block_table, self.kv_len,
                               self.rope, self.status, kv_scale, stream, self.appended)
        return q_rot

    def attention(self, q, k_cache, v_cache, block_table, cu_len, cu_len_host, kv_len_host, stream=None):
        """The newest tokens' outputs, of as many as the last ``append`` put into the cache at
        most: those of a sequence to which it appended nothing are left as they were."""
        T = q.shape[0]
        p = chunk_params(q, k_cache, v_cache, block_table, cu_len, self.kv_len, cu_len_host, kv_len_host, self.out[:T],
                         self.lse[:T], self.status, self.scale, self.window, self.sinks, self.appended)
        need = tree_chunk_attn_workspace_size(p)
        if need == 0:
            raise ValueError("tree_chunk_attn_fwd would reject these arguments")
        tree_chunk_attn_fwd(p, _grown(self, "ws_attn", need, stream), stream)
        return self.out[:T]

    def run(self, q, k, v, cu_len, cu_len_host, prefix_len, prefix_len_host, k_cache, v_cache, block_table, stream=None):
        """append, then attention: the tokens' outputs [T, Hq, D].  ``*_host`` are the
        host's copies of cu_len and prefix_len."""
        cu = np.asarray(cu_len_host, np.int32)
        kv_host = np.asarray(prefix_len_host, np.int32) + (cu[1:] - cu[:-1])
        q = self.append(q, k, v, cu_len, prefix_len, k_cache, v_cache, block_table, stream=stream)
        return self.attention(q, k_cache, v_cache, block_table, cu_len, cu, kv_host, stream)

    def score(self, logits, tokens, rows=None, temperature: float = 1.0, top: int = 0, stream=None) -> _Scores:
        """Log probabilities of ``tokens`` [R] under ``logits`` rows (those of ``rows``, or the
        first R)."""
        with _on(stream, self.device):
            out = _Scores(tokens.shape[0], top, self.device)
        tree_token_logprobs(logits, tokens, out.logprob, out.entropy, out.top_ids, out.top_logprobs, rows=rows,
                            temperature=temperature, stream=stream)
        return out
