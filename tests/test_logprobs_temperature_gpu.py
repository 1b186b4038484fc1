"""Log probabilities at the ends of the temperatures that the call takes: past 2^126, where 1 / temperature is subnormal and a
row's tokens are all alike, and near 0, where the largest has it all."""
import numpy as np
import pytest
import torch

from tests.test_logprobs_gpu import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_attention_speculative_gb300 import _build
    _build.build()


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("temperature", [3.4e38, 3e38, 1e38, 1e30, 1000.0, 1e-3, 1e-30])
def test_of_either_end(temperature, half):
    V = 5000
    x = torch.randn(4, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)) * 3
    x[1, ::7] = -float("inf")
    x[2] = -float("inf")
    got = check(x.bfloat16() if half else x, [3, 4999, 0, 17], 5, temperature=temperature)
    if temperature > 1e29:  # by the definition itself
        assert np.abs(got["lp"][[0, 3]] + np.log(V)).max() <= 2.0 ** -15 + 2.0 ** -22 * np.log(V)
        assert abs(got["ent"][0] - np.log(V)) <= 2.0 ** -15 + 2.0 ** -22 * np.log(V)
