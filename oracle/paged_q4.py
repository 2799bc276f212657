"""Float64 reference of the 4-bit cache: blocks of 32 elements as a power of two and 4-bit codes.

From the definition in include/paged_q4.h, by comparing with every power and every value. Shares no
code with the GPU path.
"""
from __future__ import annotations

import numpy as np

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def block(x):
    """(codes [32], byte) of one block of 32 numbers."""
    x = np.asarray(x, np.float64)
    if not np.isfinite(x).all():
        return np.zeros(32, np.uint8), 255
    top = np.abs(x).max()
    e = next((e for e in range(-126, 126) if top <= 6.0 * 2.0 ** e), 125)
    codes = np.empty(32, np.uint8)
    for i, v in enumerate(x):
        gap = np.abs(abs(v) / 2.0 ** e - VALUES)
        near = np.flatnonzero(gap == gap.min())
        code = near[0] if len(near) == 1 or near[0] % 2 == 0 else near[1]
        codes[i] = code | (8 if np.signbit(v) else 0)
    return codes, e + 127


def quantise(x):
    """Rows [..., D] as codes [..., D / 2] and scales [..., D / 32], both uint8."""
    x = np.asarray(x, np.float64)
    rows = x.reshape(-1, 32)
    codes, scales = np.empty(rows.shape, np.uint8), np.empty(len(rows), np.uint8)
    for i, r in enumerate(rows):
        codes[i], scales[i] = block(r)
    codes = codes.reshape(*x.shape[:-1], x.shape[-1] // 2, 2)
    return codes[..., 0] | codes[..., 1] << 4, scales.reshape(*x.shape[:-1], x.shape[-1] // 32)


def values(codes, scales):
    """The numbers that codes [..., D / 2] and scales [..., D / 32] stand for."""
    codes = np.asarray(codes)
    both = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    x = VALUES[both & 7] * np.where(both & 8, -1.0, 1.0)
    power = np.where(scales == 255, np.nan, 2.0 ** (np.asarray(scales, np.float64) - 127))
    return x * np.repeat(power, 32, -1)
