"""More of tree_attn_fwd_q8 on the GPU: tensors on the wrong device, the sum of the rounded
weights, rows beside other rows, and values at the ends of the format."""
import numpy as np
import pytest
import torch

import workloads as W
from tests.gpu_util import to_dev
from tests.q8_util import codes_dev, quantised_pools

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_attention_speculative_gb300 import _build
    _build.build()


@pytest.mark.parametrize("name", ["q", "k_cache", "block_table", "prefix_len", "k_tree", "anc_mask", "out", "lse", "status"])
def test_a_tensor_on_the_host_is_refused(name):
    import tree_attention_speculative_gb300 as ts
    case = W.build_case("host", 3, W.tree_chain(5), [40], Hq=4, Hkv=2, D=64, bs=16, permute=False)
    kc, vc, sc = quantised_pools(case)
    t = to_dev(case)
    a = dict(q=t["q"], k_cache=codes_dev(kc), v_cache=codes_dev(vc), block_table=t["block_table"], prefix_len=t["prefix_len"],
             prefix_len_host=case.prefix_len, k_tree=t["k_tree"], v_tree=t["v_tree"],
             anc_mask=torch.zeros(1, 5, 1, dtype=torch.int64, device="cuda"), pos=None, out=torch.zeros_like(t["q"]),
             lse=torch.zeros(1, 5, 4, device="cuda"), status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    ws, scales = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda"), torch.from_numpy(sc).cuda()
    ts.tree_attn_fwd_q8(ts.attn_params(**a), scales, ws)
    a[name] = a[name].cpu()
    with pytest.raises(ts.TreeSpecError):
        ts.tree_attn_fwd_q8(ts.attn_params(**a), scales, ws)
    torch.cuda.synchronize()


def _call(case, pools, mask=None, scale=0.0):
    """out and lse [B, N, Hq, ..] of one call on the case's queries over the given pools."""
    import oracle
    import tree_attention_speculative_gb300 as ts
    t = to_dev(case)
    if mask is None:
        mask = oracle.tree.build_ancestry(case.parent, case.prefix_len)[0]
    anc = torch.from_numpy(mask.view(np.int64)).cuda()
    out = torch.full(t["q"].shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full(t["q"].shape[:3], float("nan"), device="cuda")
    status = torch.zeros(case.B, dtype=torch.int32, device="cuda")
    kc, vc, sc = codes_dev(pools[0]), codes_dev(pools[1]), torch.from_numpy(pools[2]).cuda()
    p = ts.attn_params(t["q"], kc, vc, t["block_table"], t["prefix_len"], case.prefix_len, t["k_tree"], t["v_tree"], anc,
                       None, out, lse, status, scale=scale)
    ws = torch.zeros(ts.tree_attn_q8_workspace_size(p), dtype=torch.uint8, device="cuda")
    ts.tree_attn_fwd_q8(p, sc, ws)
    assert status.cpu().tolist() == [0] * case.B
    return out, lse


# (units of at most 8 rows of 128 have a kernel of their own)
@pytest.mark.parametrize("N,Hq,D", [(8, 4, 128), (30, 2, 64), (2, 4, 128), (8, 1, 128)])
@pytest.mark.parametrize("change", ["hot key late", "hot key first", "hot own key", "NaN"])
def test_a_row_does_not_depend_on_its_neighbours(N, Hq, D, change):
    """One query of the last node meets a key far above the others, or holds a NaN: every other
    row keeps its bits."""
    from oracle.attention import bf16_to_f64
    case = W.build_case("alone", 5, W.tree_chain(N), [1000], Hq=Hq, Hkv=1, D=D, bs=16, permute=False)
    pools = quantised_pools(case)
    out, lse = _call(case, pools)
    at = {"hot key late": 700, "hot key first": 3, "hot own key": None, "NaN": None}[change]
    if at is not None:   # a logit of 60
        k = bf16_to_f64(case.k_cache[case.block_table[0, at // 16], 0, at % 16])
    else:
        k = bf16_to_f64(case.k_tree[0, N - 1, 0])
    q = k * 60.0 / (case.scale * (k * k).sum())
    if change == "NaN":
        q[0] = np.nan
    case.q[0, N - 1, Hq - 1] = W.bf16_bits(q.astype(np.float32))
    out2, lse2 = _call(case, pools)
    others = np.ones((N, Hq), bool)
    others[N - 1, Hq - 1] = False
    assert torch.equal(out[0][others], out2[0][others]) and torch.equal(lse[0][others], lse2[0][others])
    assert not torch.equal(out[0, N - 1, Hq - 1], out2[0, N - 1, Hq - 1])
    assert torch.isnan(out2[0, N - 1, Hq - 1]).all() == (change == "NaN")


@pytest.mark.parametrize("B,N,Hq,D,P", [(1, 8, 4, 128, 9000), (1, 30, 4, 64, 5000), (1, 130, 4, 128, 7000), (1, 2, 4, 128, 9000)])
def test_channels_far_apart_across_the_parts_of_a_chain(B, N, Hq, D, P):
    """Even tokens hold channels of about 2^20 only, odd ones the others, of about 2^-20: every
    channel is as exact as if it were alone."""
    import oracle
    from tests.test_attn_q8_gpu import check
    case = W.build_case("apart", 9, W.tree_chain(N), [P] * B, Hq=Hq, Hkv=1, D=D, bs=16, permute=False)
    v = oracle.attention.bf16_to_f64(case.v_cache)
    small = np.arange(D) % 2 == 1
    v[:, :, 0::2] *= np.where(small, 0.0, 2.0 ** 20)
    v[:, :, 1::2] *= np.where(small, 2.0 ** -20, 0.0)
    case.v_cache = W.bf16_bits(v.astype(np.float32))
    t = oracle.attention.bf16_to_f64(case.v_tree) * np.where(small, 2.0 ** -20, 2.0 ** 20)
    case.v_tree = W.bf16_bits(t.astype(np.float32))
    pools = quantised_pools(case)
    out, lse = _call(case, pools)
    check(case, out.double().cpu().numpy(), lse.double().cpu().numpy())


@pytest.mark.parametrize("N,Hq,D", [(8, 4, 128), (30, 2, 64), (2, 4, 128)])
@pytest.mark.parametrize("scale", [1e-3, 1e-9, 1e-30, 1e-42])
def test_queries_and_scales_that_leave_no_logit(N, Hq, D, scale):
    """Zero and tiny queries, and softmax scales whose product with theirs is below fp32's range:
    every key weighs the same, and masked ones nothing."""
    import oracle
    from tests.test_attn_q8_gpu import check
    case = W.build_case("flat", 9, W.tree_chain(N), [0, 77, 500], Hq=Hq, Hkv=1, D=D, bs=16, permute=False)
    case.q[:, 0] = 0
    q = oracle.attention.bf16_to_f64(case.q[:, 1]) * 2.0 ** -120
    case.q[:, 1] = W.bf16_bits(q.astype(np.float32))
    case.scale = float(np.float32(scale))
    pools = quantised_pools(case)
    out, lse = _call(case, pools, scale=scale)
    check(case, out.double().cpu().numpy(), lse.double().cpu().numpy())


@pytest.mark.parametrize("N,Hq,D", [(8, 4, 128), (30, 2, 64), (2, 4, 128), (7, 1, 128)])
@pytest.mark.parametrize("P", [1000, 9000])
def test_outputs_are_divided_by_the_sum_of_the_rounded_weights(N, Hq, D, P):
    """One key of the prefix weighs 2^20 (1 + 0.97 / 256) times any other, which bf16 rounds down by
    nearly half a step.  Every value is 1.875, so the output is, whatever the weights; divided by the
    sum of the unrounded ones it would be a step of bf16 less.  (Chunks whose rounding is not counted
    hold less than 2^-6 of the weight: 2^-14 of the output, and a half step is 2^-9 of 1.875.)"""
    at = [300 + 7 + 65 * i if P == 1000 else P - 1 - 331 * i for i in range(10)]  # both halves, odd and even tiles
    case = W.build_case("rounded", 9, W.tree_chain(N), [P] * len(at), Hq=Hq, Hkv=1, D=D, bs=16, permute=False)
    for x, v in ((case.q, 0), (case.k_cache, 0), (case.k_tree, 0), (case.v_cache, 0x3FF0), (case.v_tree, 0x3FF0)):
        x[...] = v
    case.q[..., 0] = 0x3F80
    for b, t in enumerate(at):
        case.k_cache[case.block_table[b, t // 16], 0, t % 16, 0] = 0x4100  # 8.0; the other keys 0
    weight = 2.0 ** 20 * (1 + 0.97 / 256)
    bf16 = lambda x: float(torch.tensor(x, dtype=torch.float64).bfloat16())  # noqa: E731
    assert bf16(bf16(weight) / weight * 1.875) != 1.875
    out, lse = _call(case, quantised_pools(case), scale=float(np.log(weight) / 8))
    assert (out == 1.875).all()
    want = np.log(weight + P - 1 + np.arange(1, N + 1))
    assert (np.abs(lse.double().cpu().numpy() - want[None, :, None]) <= 2.0 ** -17 * want.max()).all()


@pytest.mark.parametrize("N", [1, 9])
def test_values_of_the_smallest_scales(N):
    """One prefix token takes all the weight: its V row as bf16, whose smallest step is 2^-133."""
    import oracle
    scales = [1, 2, 3, 4]
    codes = np.arange(256, dtype=np.uint8).reshape(2, 128)
    codes = np.where((codes & 0x7F) == 0x7F, 0, codes)
    case = W.build_case("small", 3, W.tree_chain(N), [1] * 8, Hq=1, Hkv=1, D=128, bs=16, permute=False)
    case.q[:], case.k_tree[:] = 0x3F80, 0xC1A0          # 1.0 and -20: logits of -226 for the nodes
    pools = [np.full(case.k_cache.shape, 0x38, np.uint8), np.zeros(case.v_cache.shape, np.uint8),
             np.full(case.v_cache.shape[:3] + (2,), 127, np.uint8)]
    want = np.empty((8, 128))
    for b in range(8):
        blk = case.block_table[b, 0]
        pools[1][blk, 0, 0], pools[2][blk, 0, 0, 1] = codes[b % 2], scales[b // 2]
        want[b] = oracle.cache_q8.values(codes[b % 2][None], np.array([scales[b // 2]], np.uint8))[0]
    out, _ = _call(case, pools)
    want = np.round(want * 2.0 ** 133) * 2.0 ** -133    # (np.round: halves to even)
    np.testing.assert_array_equal(out.double().cpu().numpy()[:, 0, 0], want)


@pytest.mark.parametrize("N,Hq,D", [(8, 4, 128), (30, 2, 64), (2, 4, 128)])
def test_the_largest_values_and_keys(N, Hq, D):
    """Values up to 2^87 / (P + N) under weights that pass 2^37, and keys up to 2^110."""
    import oracle
    from tests.test_attn_q8_gpu import check
    f64 = oracle.attention.bf16_to_f64
    P = 1000
    case = W.build_case("large", 9, W.tree_chain(N), [P], Hq=Hq, Hkv=1, D=D, bs=16, permute=False)
    top = 2.0 ** (87 - 11)
    for name in ("v_cache", "v_tree"):
        x = np.minimum(np.abs(f64(getattr(case, name))) / 4, 1.0) * top
        setattr(case, name, W.bf16_bits(x.astype(np.float32)))
    case.q[:], case.k_tree[:], case.k_cache[:] = 0x3F80, 0, 0
    late = np.arange(200, P)                            # their logits: 26
    case.k_cache[case.block_table[0, late // 16], 0, late % 16] = W.bf16_bits(np.float32([26.0 / (D * case.scale)]))[0]
    out, lse = _call(case, quantised_pools(case))
    check(case, out.double().cpu().numpy(), lse.double().cpu().numpy())
    case = W.build_case("large", 9, W.tree_chain(N), [P], Hq=Hq, Hkv=1, D=D, bs=16, permute=False)
    for name, e in (("k_cache", 107), ("k_tree", 107), ("q", -107)):
        x = np.clip(f64(getattr(case, name)), -8, 8) * 2.0 ** e
        setattr(case, name, W.bf16_bits(x.astype(np.float32)))
    out, lse = _call(case, quantised_pools(case))
    check(case, out.double().cpu().numpy(), lse.double().cpu().numpy())
