"""8-bit integer rows, in 64 bits on the CPU: the format from its definition,
without the library's arithmetic.

A row's scale is its largest magnitude over 127, rounded to 32 bits; an
element becomes the integer nearest to its quotient by that scale (ties to the
even one), within 127 either way.  A row with an infinity or a NaN has a NaN
scale and codes 0."""
from __future__ import annotations

import numpy as np


def quantize(x):
    """(codes [rows, cols] as int8, scales [rows] as float32) of x."""
    x = np.asarray(x, np.float64)
    codes = np.zeros(x.shape, np.int8)
    scales = np.full(x.shape[0], np.nan, np.float32)
    for r, row in enumerate(x):
        if not np.isfinite(row).all():
            continue
        scales[r] = np.float32(np.float32(np.abs(row).max()) / np.float32(127))
        s = float(scales[r])
        if s == 0:
            continue
        # numbers of 24 bits: a quotient in 64 bits is a half exactly where the true one is
        q = row / s
        low = np.floor(q)
        above = q - low
        n = low + ((above > 0.5) | ((above == 0.5) & (low % 2 == 1)))
        codes[r] = np.clip(n, -127, 127).astype(np.int8)
    return codes, scales


def values(codes, scales):
    """What codes under their rows' scales stand for, in 64 bits."""
    return np.asarray(codes, np.float64) * np.asarray(scales, np.float64)[..., None]
