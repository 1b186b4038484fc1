"""The prompt path as it is used: chunks of prompts appended and attended, decoded tokens, trees verified over the same
cache, their paths committed and scored; each step against the oracles on the whole sequences."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from tests.prompt_util import NAN, assert_rows, bf, dev, f64

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, BS, V = 3, 8, 2, 128, 16, 1000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_attention_speculative_gb300 import _build
    _build.build()


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4)])
def test_prompts_decoding_and_trees_over_one_cache(window, sinks):
    import tree_attention_speculative_gb300 as ts
    from tree_attention_speculative_gb300.step import PromptStep, TreeVerifyStep
    cfg = ts.RopeConfig(theta=500000.0)
    top = 400
    need = -(-top // BS)
    nblk = B * need
    table = np.random.default_rng(1).permutation(nblk).reshape(B, need).astype(np.int32)
    k_cache, v_cache = (bf(np.full((nblk, HKV, BS, D), NAN, np.uint16)) for _ in range(2))
    td = dev(table)
    prompt = PromptStep(B, 256, HQ, HKV, D, cfg, window=window, sinks=sinks)
    length = np.zeros(B, np.int32)
    seed = 0
    for lens in ([130, 1, 64], [0, 99, 37], [1, 1, 1], [20, 1, 0]):
        seed += 1
        cu = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
        T = int(cu[-1])
        x = W.normal_bf16(seed, "x", (T, HQ + 2 * HKV, D))
        xd = bf(x)
        out = prompt.run(xd[:, :HQ], xd[:, HQ:HQ + HKV], xd[:, HQ + HKV:], dev(cu), cu, dev(length), length, k_cache, v_cache,
                         td)
        torch.cuda.synchronize()
        length = length + np.array(lens, np.int32)
        assert prompt.kv_len.cpu().tolist() == length.tolist() and prompt.status.cpu().tolist() == [0] * B
        # the rotated queries and the cache as the append left them (checked in its own tests) are the attention's inputs
        bits = [t.view(torch.int16).cpu().numpy().view(np.uint16) for t in (prompt.q_rot[:T], k_cache, v_cache)]
        live = [np.where(c == NAN, 0, c) for c in bits[1:]]
        ref = oracle.window.chunk_attention(bits[0], *live, table, cu, length, window=window, sinks=sinks)
        mag, _ = oracle.window.chunk_attention(bits[0], live[0], live[1] & 0x7FFF, table, cu, length, window=window, sinks=sinks)
        assert_rows(f64(out), f64(prompt.lse[:T]), *ref, mag)
        # and the last row's own key, turned, is where its position says
        f = oracle.rope.frequencies(D, cfg.theta)
        b = int(np.flatnonzero(lens)[-1])
        p = length[b] - 1
        want = oracle.rope.rotate(oracle.attention.bf16_to_f64(x[cu[b + 1] - 1:cu[b + 1], HQ:HQ + HKV]), [p], D, f)[0]
        got = oracle.attention.bf16_to_f64(bits[1][table[b, p // BS], :, p % BS])
        assert np.abs(got - want).max() <= 2.0 ** -6

    # scores of the next tokens under the chunk's logits
    logits = torch.randn(5, V, device="cuda")
    s = prompt.score(logits, dev(np.array([1, 2, 3], np.int32)), rows=dev(np.array([4, 0, -1], np.int32)), top=3)
    want = oracle.logprobs.score(logits.cpu().numpy(), [1, 2, 3], [4, 0, -1], top=3)
    np.testing.assert_allclose(s.logprob.cpu()[:2], want[0][:2], atol=2.0 ** -14)
    np.testing.assert_array_equal(s.top_ids.cpu()[:2], want[2][:2])
    assert s.logprob[2].item() == 0 and s.top_ids[2].tolist() == [-1] * 3

    # two rounds of trees over that cache
    for round_ in range(2):
        seed += 1
        parent = np.stack([W.tree_random_levels(W.rng(seed, f"t{b}"), 12, 4) for b in range(B)])
        c = W.build_case("p", seed, parent, length, HQ, HKV, D, BS, True, vocab=V, plant_len=3)
        step = TreeVerifyStep(B, c.N, HQ, HKV, D, length, vocab=V, max_depth=6, rope=cfg, window=window, sinks=sinks)
        plen, new = dev(length), torch.zeros(B, dtype=torch.int32, device="cuda")
        q, kt, vt = bf(c.q), bf(c.k_tree), bf(c.v_tree)
        logits = torch.from_numpy(c.logits).cuda()
        step.run(dev(c.parent), plen, q, k_cache, v_cache, td, kt, vt, dev(c.draft), logits)
        torch.cuda.synchronize()
        bits = [t.view(torch.int16).cpu().numpy().view(np.uint16) for t in (step.q_rot, k_cache, v_cache, step.k_rot)]
        live = [np.where(a == NAN, 0, a) for a in bits[1:3]]
        tree = (bits[0], *live, table, length, bits[3])
        w = window or 1 << 20
        ref = oracle.window.tree_attention(*tree, c.v_tree, c.parent, w, sinks)
        mag, _ = oracle.window.tree_attention(*tree[:2], live[1] & 0x7FFF, *tree[3:], c.v_tree & 0x7FFF, c.parent, w, sinks)
        assert_rows(f64(step.out), f64(step.lse), *ref, mag)
        acc, L = step.accepted.cpu().numpy(), step.accept_len.cpu().numpy()
        assert L.tolist() == [3] * B
        # the emitted tokens' log probabilities: three drafts and the bonus
        s = step.logprobs(dev(c.draft), logits, top=2)
        torch.cuda.synchronize()
        lp, ids = s.logprob.cpu().numpy().reshape(B, 7), s.top_ids.cpu().numpy().reshape(B, 7, 2)
        for b in range(B):
            for d in range(4):
                node = acc[b, d]
                tok = c.draft[b, acc[b, d + 1]] if d < 3 else step.bonus[b].item()
                row, _ = oracle.logprobs.row(c.logits[b, node])
                assert abs(lp[b, d] - row[tok]) <= 2.0 ** -14
                assert ids[b, d, 0] == tok  # greedy: the token is its row's first alternative
            assert (lp[b, 4:] == 0).all() and (ids[b, 4:] == -1).all()
        step.commit(kt, vt, plen, k_cache, v_cache, td, new)
        torch.cuda.synchronize()
        assert step.status.cpu().tolist() == [0] * B
        length = length + 4
        assert new.cpu().tolist() == length.tolist()


def test_prompts_into_the_8bit_cache_are_read_by_its_attention():
    """append with scale bytes, then a tree over that cache."""
    import tree_attention_speculative_gb300 as ts
    from tests.gpu_util import ATOL, RTOL
    from tree_attention_speculative_gb300.step import PromptStep, TreeVerifyStep
    cfg = ts.RopeConfig()
    lens = np.array([70, 5, 130], np.int32)
    need = 10
    table = np.random.default_rng(2).permutation(B * need).reshape(B, need).astype(np.int32)
    kc, vc = (torch.full((B * need, HKV, BS, D), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    sc = torch.full((B * need, HKV, BS, 2), 255, dtype=torch.uint8, device="cuda")
    cu = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
    x = bf(W.normal_bf16(40, "x", (int(cu[-1]), HQ + 2 * HKV, D)))
    prompt = PromptStep(B, 256, HQ, HKV, D, cfg)
    prompt.append(None, x[:, HQ:HQ + HKV], x[:, HQ + HKV:], dev(cu), torch.zeros(B, dtype=torch.int32, device="cuda"), kc, vc,
                  dev(table), kv_scale=sc)
    torch.cuda.synchronize()
    assert prompt.kv_len.cpu().tolist() == lens.tolist()
    parent = np.stack([W.tree_random_levels(W.rng(41, f"t{b}"), 9, 3) for b in range(B)])
    c = W.build_case("p", 41, parent, lens, HQ, HKV, D, BS, True)
    step = TreeVerifyStep(B, c.N, HQ, HKV, D, lens)
    step.run(dev(c.parent), dev(lens), bf(c.q), kc, vc, dev(table), bf(c.k_tree), bf(c.v_tree), kv_scale=sc)
    torch.cuda.synchronize()
    codes, s = (t.view(torch.uint8).cpu().numpy() for t in (kc, sc)), None
    kb, sb = codes
    vb = vc.view(torch.uint8).cpu().numpy()
    vals = []
    for cb, w in ((kb, 0), (vb, 1)):
        y = oracle.cache_q8.values(cb, np.where(sb[..., w] == 255, 127, sb[..., w]))
        vals.append(W.bf16_bits(np.nan_to_num(y).astype(np.float32)))
    ref, _ = oracle.attention.tree_attention(c.q, vals[0], vals[1], table, lens, c.k_tree, c.v_tree, c.parent)
    got = f64(step.out)
    assert (np.abs(got - ref) <= ATOL + RTOL * np.abs(ref)).all()


def test_a_chunk_may_not_mix_devices():
    import tree_attention_speculative_gb300 as ts
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    a = dict(q=z(2, 4, 64), k_cache=z(3, 2, 16, 64), v_cache=z(3, 2, 16, 64), block_table=i(1, 3), cu_len=i(2), kv_len=i(1),
             cu_len_host=[0, 2], kv_len_host=[9], out=z(2, 4, 64))
    ts.chunk_params(**a)
    for name in ("q", "v_cache", "kv_len", "out"):
        with pytest.raises(ts.TreeSpecError):
            ts.chunk_params(**{**a, name: a[name].cpu()})
    with pytest.raises(ts.TreeSpecError):
        ts.tree_chunk_attn_fwd(ts.chunk_params(**a), torch.zeros(1 << 16, dtype=torch.uint8))


@pytest.mark.parametrize("as_handle", [False, True])
def test_a_step_on_another_stream_while_the_current_one_is_busy(as_handle):
    """What a step makes for a call (its workspace, the scores) is filled on the call's stream."""
    import tree_attention_speculative_gb300 as ts
    from tree_attention_speculative_gb300.step import PromptStep
    lens, V = np.array([3, 40], np.int32), 1000
    cu = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
    T, past = int(cu[-1]), np.array([700, 90], np.int32)
    table = dev(np.arange(2 * 60, dtype=np.int32).reshape(2, 60))
    x = bf(W.normal_bf16(50, "x", (T, HQ + 2 * HKV, D)))
    logits, tokens = torch.randn(T, V, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda")
    pools = [bf(W.normal_bf16(51, n, (120, HKV, BS, D))) for n in "kv"]
    side = torch.cuda.Stream()
    got = []
    for stream in (side.cuda_stream if as_handle else side, None):
        step = PromptStep(2, T, HQ, HKV, D, ts.RopeConfig())
        k_cache, v_cache = (p.clone() for p in pools)
        cud, pastd = dev(cu), dev(past)
        torch.cuda.synchronize()
        if stream is not None:
            torch.cuda._sleep(50_000_000)
        out = step.run(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], cud, cu, pastd, past, k_cache, v_cache, table, stream=stream)
        s = step.score(logits, tokens, top=3, stream=stream)
        side.synchronize()
        torch.cuda.synchronize()
        got.append((out, step.lse, s.logprob, s.entropy, s.top_ids, s.top_logprobs))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert (got[0][2] < 0).all()
