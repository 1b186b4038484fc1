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
