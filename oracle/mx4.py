"""Plain float64 definition of microscaled 4-bit floating point (test infrastructure only;
see the package docstring for who may import it).

Source: the OCP Microscaling Formats (MX) specification v1.0, FP4 (e2m1 elements, e8m0 scales
of 32 elements) with its conversion: the shared exponent is floor(log2 of the block's largest
magnitude) less 2, the exponent of the largest code.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx4_scale_index(rows: int, k: int) -> np.ndarray:
    """Byte of the scale tiles that holds block b of row r, as [rows][k / 32]."""
    r, b = np.arange(rows)[:, None], np.arange(k // BLOCK)[None]
    return ((r // 128) * -(-k // 128) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4


def mx4_quantize(x):
    """(codes [rows][k / 2], scales [tiles]) as uint8 of x [rows][k]."""
    x = np.asarray(x, dtype=np.float64)
    rows, k = x.shape
    blk = x.reshape(rows, k // BLOCK, BLOCK)
    top = np.max(np.abs(blk), axis=2)
    bad = ~np.isfinite(top)
    # frexp: top = f * 2^e, f in [0.5, 1), so floor(log2 top) = e - 1
    e = np.where(top > 0, np.frexp(np.where(bad, 1.0, top))[1] - 1 - 2, -127)
    e = np.clip(e, -127, 127)
    a = np.where(bad[:, :, None], 0.0, blk) * np.exp2(-e.astype(np.float64))[:, :, None]
    dist = np.abs(np.abs(a)[..., None] - MAGNITUDES)
    near = dist == dist.min(axis=-1, keepdims=True)
    lo = near.argmax(axis=-1)                        # the lower of the nearest codes
    tie = near.sum(axis=-1) > 1
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo) + 8 * np.signbit(a)
    code = code.reshape(rows, k).astype(np.uint8)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    scales = np.zeros(-(-rows // 128) * -(-k // 128) * 512, dtype=np.uint8)
    scales[mx4_scale_index(rows, k)] = np.where(bad, 255, e + 127)
    return codes, scales


def mx4_values(codes, scales) -> np.ndarray:
    """The float64 values [rows][k] that codes and scales stand for."""
    codes = np.asarray(codes)
    rows, k = codes.shape[0], 2 * codes.shape[1]
    c = np.empty((rows, k), dtype=np.int64)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    s = np.asarray(scales).reshape(-1)[mx4_scale_index(rows, k)].astype(np.float64)
    s = np.where(s == 255, np.nan, np.exp2(s - 127)).repeat(BLOCK, axis=1)
    return np.where(c >= 8, -1.0, 1.0) * MAGNITUDES[c % 8] * s
