"""Helpers of the 8-bit cache tests: pools on the host and the device, and their
values in the form the bf16 oracle takes."""
import numpy as np
import torch

import oracle
import workloads as W


def quantised_pools(case):
    """The case's bf16 pools as e4m3 codes and scale bytes [blocks, Hkv, bs, 2] (host),
    and in their place in the case the bf16 bits of what those stand for (a 4-bit
    significand times a power of two: exact in bf16)."""
    out, scales = [], []
    for name in ("k_cache", "v_cache"):
        codes, s = oracle.cache_q8.quantise(oracle.attention.bf16_to_f64(getattr(case, name)))
        vals = oracle.cache_q8.values(codes, s)
        bits = W.bf16_bits(vals.astype(np.float32))
        assert (oracle.attention.bf16_to_f64(bits) == vals).all()
        setattr(case, name, bits)
        out.append(codes)
        scales.append(s)
    return out[0], out[1], np.stack(scales, axis=-1)


def codes_dev(codes):
    return torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn)


def run_q8(case, max_depth=None, pools=None, rope=None):
    """One verification step over the 8-bit pools; returns the step and its device tensors."""
    from tests.gpu_util import to_dev
    from tree_attention_speculative_gb300.step import TreeVerifyStep
    kc, vc, sc = quantised_pools(case) if pools is None else pools
    t = to_dev(case)
    t.update(k_cache=codes_dev(kc), v_cache=codes_dev(vc), kv_scale=torch.from_numpy(sc).cuda())
    step = TreeVerifyStep(case.B, case.N, case.Hq, case.Hkv, case.D, case.prefix_len, vocab=case.vocab,
                          max_depth=max_depth, rope=rope)
    step.run(t["parent"], t["prefix_len"], t["q"], t["k_cache"], t["v_cache"], t["block_table"], t["k_tree"],
             t["v_tree"], t.get("draft"), t.get("logits"), kv_scale=t["kv_scale"])
    torch.cuda.synchronize()
    return step, t
