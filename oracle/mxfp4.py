"""MXFP4 oracle, in 64 bits on the CPU: the format from its definition, value
by value, without the library's arithmetic.

A block of 32 elements has the scale 2^s, s = max(-127, floor(log2(amax)) - 2),
and each element becomes the nearest of the E2M1 numbers (ties to the even
code) times the scale; blocks with an infinity or a NaN are NaN."""
from __future__ import annotations

import math

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
ORDER = [0, 2, 4, 6, 1, 3, 5, 7]  # blocks of a chunk in the order their scale bytes are stored


def nearest_code(a: np.ndarray) -> np.ndarray:
    """Code (0..7) of the magnitude nearest to a >= 0, ties to the even code."""
    code = np.zeros(a.shape, np.int64)
    for i in range(1, 8):
        mid = (MAGNITUDES[i - 1] + MAGNITUDES[i]) / 2
        code = np.where((a > mid) | ((a == mid) & (i % 2 == 0)), i, code)
    return code


def quantize(x):
    """(codes [rows, blocks * 32] of 0..15, exponents [rows, blocks], NaN
    blocks as 128) of x [rows, cols], cols padded with zeros to 256."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    v = np.zeros((rows, -(-cols // 256) * 256))
    v[:, :cols] = x
    v = v.reshape(rows, -1, 32)
    codes = np.zeros(v.shape, np.int64)
    exps = np.zeros(v.shape[:2], np.int64)
    for r in range(rows):
        for b in range(v.shape[1]):
            blk = v[r, b]
            if not np.all(np.isfinite(blk)):
                exps[r, b] = 128
                continue
            top = np.abs(blk).max()
            s = -127 if top == 0 else max(-127, math.frexp(top)[1] - 1 - 2)
            exps[r, b] = s
            codes[r, b] = nearest_code(np.abs(blk) / 2.0 ** s) | (np.signbit(blk).astype(np.int64) << 3)
    return codes.reshape(rows, -1), exps


def stored(codes, exps):
    """Code bytes [rows, row bytes] and scale bytes [chunks, rows, 8]."""
    c = codes.astype(np.uint8)
    b = (exps + 127).astype(np.uint8).reshape(exps.shape[0], -1, 8)[:, :, ORDER]
    return c[:, 0::2] | (c[:, 1::2] << 4), np.ascontiguousarray(b.transpose(1, 0, 2))


def values(code_bytes, scale_bytes, cols):
    """What stored bytes stand for, [rows, cols] in 64 bits."""
    code_bytes, scale_bytes = np.asarray(code_bytes), np.asarray(scale_bytes)
    rows = code_bytes.shape[0]
    c = np.stack([code_bytes & 15, code_bytes >> 4], -1).reshape(rows, -1)
    s = np.zeros((rows, scale_bytes.shape[0], 8), np.int64)
    s[:, :, ORDER] = scale_bytes.transpose(1, 0, 2)
    s = s.reshape(rows, -1)
    scale = np.where(s == 255, np.nan, 2.0 ** (s - 127.0))
    v = MAGNITUDES[c & 7] * np.where(c & 8, -1.0, 1.0)
    return (v.reshape(rows, -1, 32) * scale[:, :, None]).reshape(rows, -1)[:, :cols]


def quantized_values(x):
    """The values x rounds to."""
    codes, exps = quantize(x)
    return values(*stored(codes, exps), x.shape[1])
