"""Oracle: rows of the 8-bit KV cache, by definition (test infrastructure only).

A row of values x is stored as e4m3 codes and a scale byte s, value = code *
2^(s - 127).  s is the smallest in [1, 247] with max |x| <= 448 * 2^(s - 127)
over the row (247 if it has an infinity); a code is the e4m3 value nearest
x * 2^(127 - s), ties to the even code, held within +-448.  A row with a NaN is
all NaN: s = 255 and codes of 0x7f.

The e4m3 codes themselves: sign, 4 exponent bits e (bias 7), 3 mantissa bits m:
2^(e-7) (1 + m/8), or 2^-6 (m/8) for e = 0; 0x7f and 0xff are NaN.
"""
from __future__ import annotations

import numpy as np


def _table():
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = 2.0 ** (e - 7) * (1 + m / 8) if e else 2.0 ** -6 * (m / 8)
        v[c] = np.nan if (c & 0x7F) == 0x7F else (-x if c & 0x80 else x)
    return v


E4M3 = _table()
_POS = E4M3[:0x7F]  # 0 .. 448 in order


def encode(x):
    """The code of each double (already scaled)."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    a = np.where(np.isnan(x), 0.0, a)
    hi = np.clip(np.searchsorted(_POS, a), 1, 0x7E)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def quantise(x):
    """Rows x [..., D] fp64 -> codes [..., D], scale bytes [...]."""
    x = np.asarray(x, np.float64)
    bad = np.isnan(x).any(axis=-1)
    top = np.where(np.isnan(x), 0.0, np.abs(x)).max(axis=-1)
    s = np.ones(top.shape, np.int64)
    for b in range(1, 247):
        s = np.where(top > 448.0 * 2.0 ** (b - 127), b + 1, s)
    codes = encode(x * 2.0 ** (127.0 - s[..., None]))
    return np.where(bad[..., None], 0x7F, codes).astype(np.uint8), np.where(bad, 255, s).astype(np.uint8)


def values(codes, scale):
    """What codes [..., D] and scale bytes [...] stand for, fp64."""
    return E4M3[codes] * 2.0 ** (scale.astype(np.float64)[..., None] - 127.0)
