"""TreeVerifyStep's workspaces (no GPU needed: the library's calls are replaced)."""
import numpy as np
import pytest
import torch

from tree_attention_speculative_gb300 import step as step_module


@pytest.mark.parametrize("q8", [False, True])
def test_a_workspace_that_grows_leaves_the_captured_one_alive(monkeypatch, q8):
    """A captured graph replays into the workspace it was captured with, so that memory stays the
    step's own when longer prefixes want more."""
    need, seen = [0], []
    monkeypatch.setattr(step_module, "tree_attn_workspace_size", lambda p: need[0])
    monkeypatch.setattr(step_module, "tree_attn_q8_workspace_size", lambda p: need[0])
    monkeypatch.setattr(step_module, "tree_attn_fwd", lambda p, ws, stream: seen.append(ws))
    monkeypatch.setattr(step_module, "tree_attn_fwd_q8", lambda p, sc, ws, stream: seen.append(ws))
    B, N, Hq, Hkv, D = 1, 3, 2, 1, 64
    step = step_module.TreeVerifyStep(B, N, Hq, Hkv, D, np.zeros(B, np.int32), device="cpu")
    z = lambda *s: torch.zeros(*s, dtype=torch.uint8 if q8 and len(s) == 4 and s[2] == 16 else torch.bfloat16)  # noqa: E731
    args = (z(B, N, Hq, D), z(2, Hkv, 16, D), z(2, Hkv, 16, D), torch.zeros(B, 2, dtype=torch.int32),
            torch.zeros(B, dtype=torch.int32), z(B, N, Hkv, D), z(B, N, Hkv, D))
    sc = torch.zeros(2, Hkv, 16, 2, dtype=torch.uint8) if q8 else None
    kept = {}
    for need[0] in (512, 256, 1024, 768, 5000, 5001):
        step.attention(*args, kv_scale=sc)
        ws = seen[-1]
        assert ws.numel() >= need[0] and (ws == 0).all()
        kept[ws.data_ptr()] = ws.numel()
    del ws
    addresses = [seen[i].data_ptr() for i in range(6)]
    seen.clear()
    held = {t.data_ptr() for t in step.outgrown} | {(step.ws_attn_q8 if q8 else step.ws_attn).data_ptr()}
    assert set(addresses) == held
    assert sum(t.numel() for t in step.outgrown) < (step.ws_attn_q8 if q8 else step.ws_attn).numel()
