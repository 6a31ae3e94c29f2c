"""Activations in 8 bits (oracle; test infrastructure only).

e4m3: sign, 4 bits of exponent (bias 7), 3 of mantissa; 0x7f is NaN, the largest
finite value 448 = 1.75 * 2^8, the smallest normal one 2^-6, subnormal steps 2^-9.
Each block of 128 elements of a row has a scale: the smallest power of two, at
least 2^-117, with which its largest finite magnitude stays within 448 (1 where
all are zero). Magnitudes above 1.875 * 2^127 count as that, infinities and NaN
become NaN.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
MOST = 1.875 * 2.0 ** 127


def decode(codes):
    """fp64 values of e4m3 codes."""
    c = np.asarray(codes, np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


FINITE = decode(np.arange(0x7F))  # in rising order


def encode(v):
    """e4m3 codes of fp64 values within 448, to nearest, halves to the even code; NaN to 0x7f."""
    a = np.abs(v)
    hi = np.clip(np.searchsorted(FINITE, a, side="left"), 0, len(FINITE) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = FINITE[hi] - a, a - FINITE[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.isnan(v), 0x7F, code)
    return (code | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def scale_of(top):
    """The scale for a largest magnitude (an exact search over powers of two)."""
    if top == 0:
        return 1.0
    k = -117
    while top > 448.0 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def pack(x):
    """(codes, scales) of rows."""
    x = np.asarray(x, np.float64)
    rows, dim = x.shape
    codes, scales = np.zeros(x.shape, np.uint8), np.ones((rows, -(-dim // BLOCK)))
    for b in range(scales.shape[1]):
        v = x[:, b * BLOCK:(b + 1) * BLOCK]
        v = np.where(np.isinf(v), np.nan, np.clip(v, -MOST, MOST))
        top = np.where(np.isnan(v), 0.0, np.abs(v)).max(1)
        scales[:, b] = [scale_of(t) for t in top]
        codes[:, b * BLOCK:(b + 1) * BLOCK] = encode(v / scales[:, b, None])
    return codes, scales


def unpack(codes, scales):
    codes = np.asarray(codes)
    return decode(codes) * np.repeat(np.asarray(scales, np.float64), BLOCK, axis=1)[:, :codes.shape[1]]
