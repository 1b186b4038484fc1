"""Oracle: rotary positions of queries and keys, by definition in fp64 (test infrastructure only).

Pair i of the R rotated channels turns by the angle pos * f_i, f_i = theta^(-2i/R)
after scaling (see ``frequencies``), as multiplication by a unit complex number:
x + iy -> mscale * (x + iy) * exp(i * angle).  The pair is channels (i, i + R/2),
or (2i, 2i + 1) when interleaved; channels past R stay.
"""
from __future__ import annotations

import cmath
import math

import numpy as np


def frequencies(R, theta, scaling="none", factor=1.0, low_rot=1.0, high_rot=4.0, orig_len=0):
    """Radians a position of each of the R/2 pairs."""
    if scaling == "ntk" and R > 2:
        theta = theta * factor ** (R / (R - 2))
    out = []
    for i in range(R // 2):
        f = theta ** (-2.0 * i / R)
        if scaling == "linear":
            f /= factor
        elif scaling == "bands":
            turns = orig_len * f / (2 * math.pi)
            if turns <= low_rot:
                f /= factor
            elif turns < high_rot:
                g = (turns - low_rot) / (high_rot - low_rot)
                f = g * f + (1 - g) * f / factor
        out.append(f)
    return out


def rotate(x, pos, R, freq, interleaved=False, mscale=1.0):
    """x [T, H, D] fp64 at pos [T] -> fp64, one token and pair at a time."""
    y = np.array(x, np.float64, copy=True)
    for t in range(x.shape[0]):
        for i in range(R // 2):
            u = mscale * cmath.exp(1j * (int(pos[t]) * freq[i]))
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
            z = (x[t, :, a] + 1j * x[t, :, b]) * u
            y[t, :, a], y[t, :, b] = z.real, z.imag
    return y
