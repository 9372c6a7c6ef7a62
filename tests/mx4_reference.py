"""MX4 rows in numpy, straight from the definition: blocks of 32, one power-of-two scale, the nearest of eight magnitudes."""
from __future__ import annotations

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(v):
    """float array [rows, cols] (exact values) -> E2M1 codes [rows, 32 * blocks] and scale codes [rows, blocks]."""
    v = np.asarray(v, dtype=np.float64)
    rows, cols = v.shape
    blocks = -(-cols // 32)
    full = np.zeros((rows, 32 * blocks))
    full[:, :cols] = v
    neg = np.signbit(full)
    b = np.abs(full).reshape(rows, blocks, 32)
    top = b.max(2)  # NaN stays
    bad = ~np.isfinite(top)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.where((top > 0) & ~bad, np.floor(np.log2(np.where((top > 0) & ~bad, top, 1.0))), -1000)
        # log2 of a value just below a power of two may round up to it
        e = np.where((top > 0) & ~bad & (np.exp2(e) > top), e - 1, e)
    e = np.maximum(e - 2, -127)
    with np.errstate(invalid="ignore"):
        a = (b / np.exp2(e)[:, :, None])[..., None]
        dist = np.abs(a - LEVELS)
        near = dist.min(-1, keepdims=True)
        tied = dist == near                      # two levels where a value lies half way
        even = (np.arange(8) % 2 == 0)
        both = tied.sum(-1) > 1
        code = np.where(both, np.argmax(tied & even, -1), np.argmax(tied, -1))
        code = np.where(a[..., 0] >= 6, 7, code)
    code = np.where(bad[:, :, None], 0, code).reshape(rows, -1)
    sign = np.where(np.repeat(bad, 32, 1), 0, neg * 8)
    return (code + sign).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def pack(code, scale):
    """Codes and scales to the bytes of MX4 rows, filling included."""
    rows, cols = code.shape
    q = np.zeros((rows, -(-cols // 128) * 64), np.uint8)
    q[:, :cols // 2] = code[:, 0::2] | (code[:, 1::2] << 4)
    s = np.zeros((rows, -(-scale.shape[1] // 16) * 16), np.uint8)
    s[:, :scale.shape[1]] = scale
    return q, s


def values(q, s, cols):
    """float64 values that the bytes of MX4 rows stand for."""
    code = np.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)[:, :cols]
    v = np.where(code & 8, -1.0, 1.0) * LEVELS[code & 7]
    with np.errstate(invalid="ignore"):
        scale = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))
        return v * np.repeat(scale, 32, 1)[:, :cols]
