"""Pins of the rope and 8-bit cache oracles: closed forms, brute force, torch's own e4m3 cast."""
import math

import numpy as np
import pytest
import torch

from oracle import cache_q8, rope


def test_e4m3_table_and_rounding_match_torch():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(cache_q8.E4M3, codes)
    x = np.concatenate([np.linspace(-448, 448, 40001), np.arange(-512, 513) * 2.0 ** -10,
                        (cache_q8._POS[1:] + cache_q8._POS[:-1]) / 2])  # the ties among them
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(cache_q8.encode(x.astype(np.float32).astype(np.float64)), want)


@pytest.mark.parametrize("top,byte", [(448.0, 127), (448.5, 128), (1.75, 119), (1.7578125, 120), (1.0, 119), (0.0, 1),
                                      (2.0 ** -130, 1), (float(np.finfo(np.float32).max), 247), (np.inf, 247)])
def test_scale_byte(top, byte):
    codes, s = cache_q8.quantise(np.array([[0.0, -top, top / 3]]))
    assert s.tolist() == [byte]
    if 0 < byte - 1 and np.isfinite(top):  # the smallest that fits
        assert top <= 448 * 2.0 ** (byte - 127) and (byte == 1 or top > 448 * 2.0 ** (byte - 128))


def test_special_values():
    codes, s = cache_q8.quantise(np.array([[1.0, np.inf, -np.inf, 0.0], [np.nan, 1.0, -1.0, 0.5], [2.0, 1.0, -1.0, 0.5]]))
    assert codes[0].tolist() == [0, 0x7E, 0xFE, 0] and codes[1].tolist() == [0x7F] * 4 and s.tolist() == [247, 255, 120]
    assert cache_q8.values(codes[2:], s[2:]).tolist() == [[2.0, 1.0, -1.0, 0.5]]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("R", [2, 10, 64])
def test_rope_preserves_lengths_and_relative_positions(interleaved, R):
    g = np.random.default_rng(0)
    f = rope.frequencies(R, 10000.0)
    q, k = g.standard_normal((1, 1, 64)), g.standard_normal((1, 1, 64))
    dots = []
    for shift in (0, 5, 1000):
        a = rope.rotate(q, [7 + shift], R, f, interleaved)
        b = rope.rotate(k, [3 + shift], R, f, interleaved)
        assert np.isclose((a ** 2).sum(), (q ** 2).sum()) and (a[..., R:] == q[..., R:]).all()
        dots.append((a * b).sum())
    np.testing.assert_allclose(dots, dots[0], rtol=1e-9)
    assert (rope.rotate(q, [0], R, f, interleaved) == q).all()


def test_rope_frequencies():
    f = rope.frequencies(64, 10000.0)
    assert f[0] == 1.0 and math.isclose(f[16], 0.01)
    assert rope.frequencies(64, 10000.0, "linear", 4.0)[16] == f[16] / 4
    n = rope.frequencies(64, 10000.0, "ntk", 4.0)
    assert n[0] == 1.0 and math.isclose(n[31], f[31] / 4)  # the slowest pair slows by the factor
    b = rope.frequencies(64, 10000.0, "bands", 4.0, 1.0, 4.0, 4096)
    assert b[0] == f[0] and b[31] == f[31] / 4 and all(f[i] / 4 <= b[i] <= f[i] for i in range(32))
