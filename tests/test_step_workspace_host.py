"""TreeVerifyStep.attn_workspace_bytes is the size of the call that the step makes (no GPU needed)."""
import numpy as np
import pytest
import torch

from tests.test_abi_host import ts  # noqa: F401


def _step_and_args(window, codes=False):
    from tree_attention_speculative_gb300.step import TreeVerifyStep
    B, N, Hq, Hkv, D, bs, P = 1, 5, 2, 1, 64, 16, 60000
    pool = (P // bs + 1, Hkv, bs, D)
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    cache = dict(dtype=torch.uint8) if codes else {}
    step = TreeVerifyStep(B, N, Hq, Hkv, D, np.array([P], np.int32), device="cpu", window=window, sinks=4 if window else 0)
    return step, (z(B, N, Hq, D), z(*pool, **cache), z(*pool, **cache), z(B, pool[0], dtype=torch.int32), z(B, dtype=torch.int32),
                  z(B, N, Hkv, D), z(B, N, Hkv, D)), z(*pool[:3], 2, dtype=torch.uint8)


@pytest.mark.parametrize("window", [0, 100, 4096, 1 << 20])
def test_of_a_bf16_cache(ts, window):  # noqa: F811
    step, args, _ = _step_and_args(window)
    p = step._params(*args)
    want = ts.tree_attn_window_workspace_size(p, window, 4) if window else ts.tree_attn_workspace_size(p)
    assert step.attn_workspace_bytes(*args) == want > 0
    if window:
        assert want != ts.tree_attn_workspace_size(p)  # (so the sizes of the two calls are told apart)


def test_of_an_8bit_cache(ts):  # noqa: F811
    step, args, scale = _step_and_args(0, codes=True)
    assert step.attn_workspace_bytes(*args, kv_scale=scale) == ts.tree_attn_q8_workspace_size(step._params(*args)) > 0
    step, args, scale = _step_and_args(8, codes=True)
    with pytest.raises(ValueError):
        step.attn_workspace_bytes(*args, kv_scale=scale)
