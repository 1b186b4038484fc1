"""tree_token_logprobs against the fp64 oracle; ids exactly.

A thread sums at most 256 terms one after the other, 17 joins follow: sums are off by (256 + 17) 2^-24 at most, the
exponentials by 2^-22, so a log probability (at most a few tens) by 2^-15 with its own three fp32 steps, 2^-22 of it."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_attention_speculative_gb300 import _build
    _build.build()


def call(x, tokens, top=0, rows=None, temperature=1.0, entropy=True, stream=None):
    import tree_attention_speculative_gb300 as ts
    R = len(tokens)
    o = dict(lp=torch.full((R,), 7.0, device="cuda"), ent=torch.full((R,), 7.0, device="cuda"),
             ids=torch.full((R, top), 7, dtype=torch.int32, device="cuda"), alt=torch.full((R, top), 7.0, device="cuda"))
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    ts.tree_token_logprobs(x, i32(tokens), o["lp"], o["ent"] if entropy else None, o["ids"] if top else None,
                           o["alt"] if top else None, None if rows is None else i32(rows), temperature, stream)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in o.items()}


def close(got, want):
    fine = np.isfinite(want)
    np.testing.assert_array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    assert np.isnan(got[np.isnan(want)]).all()
    d = np.abs(got[fine] - want[fine])
    assert (d <= 2.0 ** -15 + 2.0 ** -22 * np.abs(want[fine])).all(), d.max()


def check(x, tokens, top=0, rows=None, temperature=1.0):
    flat = x.reshape(-1, x.shape[-1])
    got = call(x, tokens, top, rows, temperature)
    want = oracle.logprobs.score(flat.float().cpu().numpy(), tokens, rows, temperature, top)
    out = want[2][:, 0] == -2 if top else np.isnan(want[1])  # rows out of range
    for name, w in zip(("lp", "ent", "ids", "alt"), want):
        assert (got[name][out] == 7).all()
        (np.testing.assert_array_equal if name == "ids" else close)(got[name][~out], w[~out])
    return got


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("V", [1, 2, 5, 33, 1000, 4097, 32000, 50257, 128256])
@pytest.mark.parametrize("R,top", [(3, 0), (5, 20), (2, 1), (1, 32)])
def test_matches_oracle(half, V, R, top):
    g = np.random.default_rng(V + R)
    x = (torch.randn(R, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(V)) * 3)
    x = x.bfloat16() if half else x
    if V > 40:
        x[0, V // 4:V // 2] = -float("inf")
    check(x, g.integers(0, V, R), min(top, 32), temperature=1.0 if R != 2 else 0.7)


@pytest.mark.parametrize("R", [200, 700])
def test_many_rows(R):
    g = np.random.default_rng(R)
    x = torch.randn(R, 5003, device="cuda") * 2
    check(x, g.integers(0, 5003, R), 5)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("V", [9000, 128256, 524224])
def test_ties_sorted_rows_and_columns(half, V):
    """Rows where the choice of columns can go wrong: constant ones, ones with the best values in one thread's column,
    rising and falling ones, ties across the border of the last place."""
    x = torch.randn(8, V, device="cuda").clamp(-3, 3)
    x[0] = 1.25
    x[1] = torch.arange(V, device="cuda", dtype=torch.float32) / V
    x[2] = -torch.arange(V, device="cuda", dtype=torch.float32) / V
    x[3, 5::2048 * (2 if half else 1)] = 4.0            # one column of the first CTA (and ties)
    x[4, 5::2048] = 4.0 + torch.arange(len(x[4, 5::2048]), device="cuda") / 64
    x[5] = torch.round(x[5] * 2) / 2                    # few distinct values
    x[6, :] = -float("inf")
    x[6, [3, V - 1, V // 2]] = 0.5
    x[7, V - 40:] = 5.0
    x = x.bfloat16() if half else x
    check(x, [0, V - 1, 1, 5, 7, 9, 3, V - 2], 32)
    check(x, [0, V - 1, 1, 5, 7, 9, 3, V - 2], 7)


def test_extreme_rows():
    x = torch.zeros(7, 300, device="cuda")
    x[0] = -float("inf")
    x[1] = torch.finfo(torch.float32).min               # the type's lowest value everywhere
    x[2] = torch.finfo(torch.float32).min
    x[2, 17] = 0.0
    x[3] = 1e30
    x[3, 4] = 3e38
    x[4] = -0.0
    x[4, ::3] = 0.0                                     # equal to -0: ties by index
    x[5, 1:] = -80.0
    x[6] = torch.linspace(-100, 100, 300)
    check(x, [3, 5, 17, 4, 0, 1, -1], 6)
    got = call(x, [300, -2, 1 << 30, 0, 0, 0, 0], 0)["lp"]
    assert np.isnan(got[:3]).all() and np.isfinite(got[3:]).all()


@pytest.mark.parametrize("half", [False, True])
def test_strided_unaligned_and_picked_rows(half):
    base = torch.randn(9, 6, 1111, device="cuda")
    base = base.bfloat16() if half else base
    check(base, np.arange(54) % 1111, 4)                                    # [B, N, V]
    check(base[2:, :, 3:1001].reshape(-1, 998)[:5], [1, 2, 3, 4, 5], 4)
    view = base[:, 0, 1:]                                                   # rows 6 * 1111 apart, off their alignment
    check(view, np.arange(9), 20)
    flat = base.view(54, 1111)
    check(flat, [5, 6, 7, 8, 9, 1], 3, rows=[53, 0, -1, 53, 54, 7])


def test_row_offsets_past_32_bits():
    V = 128256
    x = torch.empty(17000, V, device="cuda")
    x[-2:] = torch.randn(2, V, device="cuda")
    a = call(x, [5, 6], 8, rows=[16998, 16999])
    b = call(x[-2:].clone(), [5, 6], 8)
    for k in a:
        np.testing.assert_array_equal(a[k], b[k])


def test_repeats_in_a_graph_and_on_another_stream():
    import tree_attention_speculative_gb300 as ts
    x = torch.randn(40, 50257, device="cuda")
    t = torch.arange(40, dtype=torch.int32, device="cuda")
    first = call(x, t.cpu().numpy(), 9)
    s = torch.cuda.Stream()
    second = call(x, t.cpu().numpy(), 9, stream=s)
    lp, ids = torch.zeros(40, device="cuda"), torch.zeros(40, 9, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ts.tree_token_logprobs(x, t, lp, top_ids=ids)
    for _ in range(2):
        lp.zero_()
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(lp.cpu().numpy(), first["lp"])
        np.testing.assert_array_equal(ids.cpu().numpy(), first["ids"])
    for k in first:
        np.testing.assert_array_equal(first[k], second[k])


def test_only_some_outputs():
    import tree_attention_speculative_gb300 as ts
    x = torch.randn(3, 777, device="cuda")
    want = oracle.logprobs.score(x.cpu().numpy(), [0, 0, 0], top=2)
    ent = torch.zeros(3, device="cuda")
    ts.tree_token_logprobs(x, None, None, ent)
    ids = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    ts.tree_token_logprobs(x, None, None, top_ids=ids)
    alt = torch.zeros(3, 2, device="cuda")
    ts.tree_token_logprobs(x, None, None, top_logprobs=alt)
    close(ent.cpu().numpy(), want[1])
    np.testing.assert_array_equal(ids.cpu().numpy(), want[2])
    close(alt.cpu().numpy(), want[3])
    ts.tree_token_logprobs(x, torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(0, device="cuda"))
