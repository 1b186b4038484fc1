"""GPU parity of tree_rope with the fp64 oracle.

An output is within half a bf16 step of the exact value (2^-8 of it) plus the
fp32 error of a pair: sine and cosine to about 2^-22 of 1 (the angle's fraction
of a turn is rounded to 24 bits and sincospi is good to an ulp), two products
and a sum, so 2^-20 of the pair's length is ample."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_attention_speculative_gb300 import _build
    _build.build()


def _check(got, x, pos, cfg):
    """got, x bf16 tensors [B, N, H, D]; pos [B, N]."""
    D = x.shape[-1]
    R = cfg.rotary_dim or D
    f = oracle.rope.frequencies(R, cfg.theta, cfg.scaling, cfg.factor, cfg.low_rot, cfg.high_rot, cfg.orig_len)
    xs = x.float().cpu().numpy().astype(np.float64).reshape(-1, x.shape[2], D)
    ref = oracle.rope.rotate(xs, pos.cpu().numpy().reshape(-1), R, f, cfg.interleaved, cfg.mscale)
    y = got.float().cpu().numpy().astype(np.float64).reshape(ref.shape)
    length = cfg.mscale * np.sqrt((xs[..., :R] ** 2).max(axis=-1, keepdims=True) * 2)
    assert (np.abs(y - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * length).all()
    np.testing.assert_array_equal(y[..., R:], xs[..., R:])


def _inputs(B, N, Hq, Hkv, D, seed=0, fused=False, top=1 << 20):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, N, Hq + 2 * Hkv, D, device="cuda", generator=g).bfloat16()
    q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    pos = torch.randint(0, top, (B, N), device="cuda", generator=g, dtype=torch.int32)
    return q, k, pos


CASES = [
    # B, N, Hq, Hkv, D, rotary_dim, interleaved, fused, more
    (1, 1, 1, 1, 64, 0, False, False, {}),
    (1, 5, 2, 2, 64, 0, True, True, {}),
    (3, 37, 8, 2, 128, 0, False, True, dict(theta=500000.0, scaling="bands", factor=8.0, orig_len=8192)),
    (2, 26, 12, 3, 128, 0, True, False, dict(scaling="linear", factor=4.0)),
    (2, 7, 4, 4, 128, 32, True, True, dict(scaling="ntk", factor=16.0)),
    (2, 7, 4, 4, 128, 96, False, False, dict(scaling="bands", factor=32.0, high_rot=32.0, orig_len=4096, mscale=1.35)),
    (2, 9, 3, 1, 64, 20, False, True, {}),          # 10 pairs: no whole 16-byte chunks
    (2, 9, 3, 1, 64, 10, True, False, dict(scaling="ntk", factor=2.0)),
    (1, 4, 2, 1, 128, 2, False, False, dict(scaling="ntk", factor=2.0)),
    (1, 1, 256, 16, 128, 0, False, False, {}),
    (5, 61, 16, 1, 64, 48, False, True, {}),
]


@pytest.mark.parametrize("B,N,Hq,Hkv,D,R,inter,fused,more", CASES)
def test_rope_matches_oracle(B, N, Hq, Hkv, D, R, inter, fused, more):
    import tree_attention_speculative_gb300 as ts
    cfg = ts.RopeConfig(rotary_dim=R, interleaved=inter, **more)
    q, k, pos = _inputs(B, N, Hq, Hkv, D, seed=B * N, fused=fused)
    keep_q, keep_k = q.clone(), k.clone()
    qo = torch.full((B, N, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    ko = torch.full((B, N, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    ts.tree_rope(q, k, pos, qo, ko, cfg)
    _check(qo, keep_q, pos, cfg)
    _check(ko, keep_k, pos, cfg)
    assert torch.equal(q, keep_q) and torch.equal(k, keep_k)
    # one at a time, and (dense) in place
    q2, k2 = torch.empty_like(qo), torch.empty_like(ko)
    ts.tree_rope(q, None, pos, q2, None, cfg)
    ts.tree_rope(None, k, pos, None, k2, cfg)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    if not fused:
        ts.tree_rope(q, k, pos, q, k, cfg)
        assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("R", [128, 20])
def test_rope_extreme_positions(R):
    """Whole turns drop out exactly: the largest, the smallest and negative positions."""
    import tree_attention_speculative_gb300 as ts
    cfg = ts.RopeConfig(rotary_dim=R, theta=500000.0)
    q, k, _ = _inputs(1, 8, 4, 2, 128)
    pos = torch.tensor([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 255, 2 ** 24 + 1, 131071]], dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    ts.tree_rope(q, k, pos, qo, ko, cfg)
    _check(qo, q, pos, cfg)
    assert torch.equal(qo[0, 0], q[0, 0])


def test_rope_many_tokens_other_stream_and_graph():
    import tree_attention_speculative_gb300 as ts
    cfg = ts.RopeConfig(scaling="linear", factor=2.0)
    q, k, pos = _inputs(1, 70001, 2, 1, 64, top=70001)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ts.tree_rope(q, k, pos, qo, ko, cfg, stream=side)
    side.synchronize()
    pick = torch.randint(0, 70001, (300,), device="cuda")
    pick[:3] = torch.tensor([0, 69999, 70000])
    _check(qo[:, pick], q[:, pick], pos[:, pick], cfg)
    _check(ko[:, pick], k[:, pick], pos[:, pick], cfg)
    want = qo.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ts.tree_rope(q, k, pos, qo, ko, cfg)
    qo.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, want)


def test_step_positions_and_commits_on_the_bf16_cache():
    """TreeVerifyStep with a rope configuration is tree_rope, then the step without one; commit
    appends the rotated keys."""
    import tree_attention_speculative_gb300 as ts
    from tests.gpu_util import to_dev
    from tree_attention_speculative_gb300.step import TreeVerifyStep
    cfg = ts.RopeConfig(interleaved=True, rotary_dim=64)
    parent = np.stack([W.tree_from_widths([4, 3, 2, 1, 1])] * 2)
    case = W.build_case("roped", 3, parent, [40, 300], Hq=8, Hkv=2, D=128, bs=16, permute=True, vocab=300, plant_len=[2, 4],
                        spare_tokens=6)
    t = to_dev(case)
    pools = t["k_cache"].clone(), t["v_cache"].clone()
    a = TreeVerifyStep(2, 26, 8, 2, 128, case.prefix_len, vocab=300, max_depth=5, rope=cfg)
    a.run(t["parent"], t["prefix_len"], t["q"], *pools, t["block_table"], t["k_tree"], t["v_tree"], t["draft"], t["logits"])
    q, k = torch.empty_like(t["q"]), torch.empty_like(t["k_tree"])
    ts.tree_rope(t["q"], t["k_tree"], a.pos, q, k, cfg)
    b = TreeVerifyStep(2, 26, 8, 2, 128, case.prefix_len, vocab=300, max_depth=5)
    b.run(t["parent"], t["prefix_len"], q, *pools, t["block_table"], k, t["v_tree"], t["draft"], t["logits"])
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse) and torch.equal(a.accepted, b.accepted)
    other = pools[0].clone(), pools[1].clone()
    new, want = torch.empty_like(t["prefix_len"]), torch.empty_like(t["prefix_len"])
    a.commit(t["k_tree"], t["v_tree"], t["prefix_len"], *pools, t["block_table"], new)
    ts.tree_commit_accepted(k, t["v_tree"], b.accepted, b.accept_len, t["prefix_len"], *other, t["block_table"], want)
    assert torch.equal(pools[0], other[0]) and torch.equal(pools[1], other[1]) and torch.equal(new, want)
    assert new.cpu().tolist() == [43, 305]


def test_expanded_inputs_are_refused():
    """A token or a head that an expanded view repeats has no stride to hand over."""
    import tree_attention_speculative_gb300 as ts
    q, k, pos = _inputs(2, 6, 4, 2, 64)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    for x in (q[:1, :1].expand(2, 6, 4, 64), q[:, :1].expand(2, 6, 4, 64), q[:, :, :1].expand(2, 6, 4, 64)):
        with pytest.raises(ts.TreeSpecError):
            ts.tree_rope(x, k, pos, qo, ko, ts.RopeConfig())
    one = pos[:, :1].contiguous()
    with pytest.raises(ts.TreeSpecError):
        ts.tree_rope(q[:1, :1].expand(2, 1, 4, 64), None, one, qo[:, :1].contiguous(), None, ts.RopeConfig())
    # a single token or head may have any stride
    wide = torch.empty(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda").as_strided((1, 1, 4, 64), (0, 0, 64, 1))
    wide.copy_(q[:1, :1])
    out = torch.empty(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    ts.tree_rope(wide, None, one[:1], out, None, ts.RopeConfig())
    ts.tree_rope(q, None, pos, qo, None, ts.RopeConfig())
    assert torch.equal(out[0, 0], qo[0, 0])
