"""A prompt step of a batch in which one sequence's append fails: its error stays in ``status``, none of its rows is attended
(they are not in the cache), and the others are as they would be without it."""
import numpy as np
import pytest
import torch

import workloads as W
from tests.prompt_util import bf, dev, f64

pytestmark = pytest.mark.gpu

SHAPE, BAD_BLOCK, INVALID_TREE = -2, -5, -3
HQ, HKV, BS = 8, 2, 16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_attention_speculative_gb300 import _build
    _build.build()


class Run:
    """A step over sequences of `past` tokens with `lens` new ones, outputs of 7 before it."""

    def __init__(self, lens, past, D, window=0):
        import tree_attention_speculative_gb300 as ts
        from tree_attention_speculative_gb300.step import PromptStep
        self.lens, self.past, B = np.array(lens, np.int32), np.array(past, np.int32), len(lens)
        self.cu = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
        need = -(-int((self.lens + self.past).max() + 40) // BS)
        self.table = np.random.default_rng(3).permutation(B * need).reshape(B, need).astype(np.int32)
        T = int(self.cu[-1])
        self.x = bf(W.normal_bf16(80, "x", (T, HQ + 2 * HKV, D)))
        self.k, self.v = (bf(W.normal_bf16(81, n, (B * need, HKV, BS, D))) for n in "kv")
        self.step = PromptStep(B, T, HQ, HKV, D, ts.RopeConfig(), window=window, sinks=4 if window else 0)
        self.step.out.fill_(7.0)
        self.step.lse.fill_(7.0)

    def call(self):
        x = self.x
        out = self.step.run(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], dev(self.cu), self.cu, dev(self.past), self.past,
                            self.k, self.v, dev(self.table))
        torch.cuda.synchronize()
        return f64(out), f64(self.step.lse)


@pytest.mark.parametrize("D,window", [(128, 0), (64, 0), (128, 50)])
@pytest.mark.parametrize("past", [5, 300])  # fewer cached tokens than new ones, and more
@pytest.mark.parametrize("lens", [[33, 40, 1], [1, 40, 700]])
@pytest.mark.parametrize("fault", ["block", "status"])
def test_a_failed_append_is_not_attended(fault, lens, past, D, window):
    good = Run(lens, [200, past, 900], D, window)
    want, want_lse = good.call()
    assert good.step.status.cpu().tolist() == [0] * 3
    r = Run(lens, [200, past, 900], D, window)
    if fault == "block":
        r.table[1, past // BS + 1] = r.k.shape[0]  # past the pool, among the blocks of the new tokens
        code = BAD_BLOCK
    else:
        r.step.status[1] = code = INVALID_TREE
    for _ in range(2):  # and again, with the error still there
        got, lse = r.call()
        assert r.step.status.cpu().tolist() == [0, code, 0]
        assert r.step.kv_len.cpu().tolist() == [200 + lens[0], past, 900 + lens[2]]
        own = np.zeros(int(r.cu[-1]), bool)
        own[r.cu[1]:r.cu[2]] = True
        assert (got[own] == 7).all() and (lse[own] == 7).all()
        np.testing.assert_array_equal(got[~own], want[~own])
        np.testing.assert_array_equal(lse[~own], want_lse[~own])
        assert r.step.appended.cpu().tolist() == [lens[0], 0, lens[2]]
    # the error taken back and the block put right
    r.step.status.zero_()
    r.table = good.table
    got, lse = r.call()
    assert r.step.status.cpu().tolist() == [0] * 3 and r.step.appended.cpu().tolist() == lens
    np.testing.assert_array_equal(got, want)
    np.testing.assert_array_equal(lse, want_lse)


def test_more_rows_than_were_appended_are_refused():
    """The last rows alone may be attended; more than the append brought may not, and an error that is there is kept."""
    import tree_attention_speculative_gb300 as ts
    r = Run([30, 20], [100, 50], 128)
    want, _ = r.call()
    step, T = r.step, 50
    for lens, code in (([1, 20], [0, 0]), ([30, 20], [0, 0]), ([30, 20], [SHAPE, 0]), ([30, 20], [INVALID_TREE, 0])):
        cu = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
        q = torch.cat([step.q_rot[30 - lens[0]:30], step.q_rot[30:]])
        step.status.zero_()
        if code[0] == INVALID_TREE:
            step.status[0] = INVALID_TREE
        if code[0]:
            step.appended[0] = 29
        step.out.fill_(7.0)
        out = f64(step.attention(q, r.k, r.v, dev(r.table), dev(cu), cu, r.lens + r.past))
        assert step.status.cpu().tolist() == code
        rows = np.r_[30 - lens[0]:30, 30:50]
        live = np.arange(len(rows)) >= (lens[0] if code[0] else 0)
        # (rows that are tiled otherwise may round otherwise: each side by half a step of the output, 2^-8 of it, and by
        # 2^-8 + 2^-10 of the values for the weights, as in prompt_util.assert_rows)
        tol = 2.0 ** -7 * np.abs(want[rows]) + 2 * (2.0 ** -8 + 2.0 ** -10) * np.abs(f64(r.v)).max()
        assert (np.abs(out - want[rows]) <= tol)[live].all()
        assert (out[~live] == 7).all()
