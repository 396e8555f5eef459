"""Plain CPU oracle of the block-scaled e4m3 format, its products, and the RMS
norm: the definitions written down in numpy, sharing no code with the CUDA
library. TEST INFRASTRUCTURE ONLY.

The format fixes three steps to fp32 (the scale, its reciprocal, the scaled
value), which numpy float32 takes with one IEEE rounding each; the rounding to
e4m3 is an argmin over the exactly decoded code values; everything else is
fp64.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
MIN_AMAX = np.float32(2.0 ** -117)


def e4m3_values() -> np.ndarray:
    """fp64 value of every code 0..255: sign bit 7, exponent bits 6-3 (bias 7,
    0 subnormal), mantissa bits 2-0; codes 0x7f and 0xff are NaN."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        mag = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if (c & 127) == 127 else (-mag if c & 128 else mag)
    return v


VALUES = e4m3_values()


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """Codes of fp32 values: nearest magnitude, ties to the even code,
    saturating at 448; the sign bit is kept; NaN gives 0x7f."""
    x = np.asarray(x, np.float32)
    mags = VALUES[:127]
    mid = (mags[1:] + mags[:-1]) / 2                    # exact in fp64
    a = np.abs(x.astype(np.float64))
    lo = np.searchsorted(mid, a, side="left")           # a tie gets the lower code
    up = np.searchsorted(mid, a, side="right")          # and here the upper one
    mag = np.where(lo % 2 == 0, lo, up)
    code = (mag | np.where(np.signbit(x), 128, 0)).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(127), code)


def _block_index(n: int, size: int) -> np.ndarray:
    return np.arange(n) // size


def quantize(x: np.ndarray, block_rows: int):
    """(codes uint8 [rows, cols], scale float32) of fp32 values."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    rb, cb = -(-rows // block_rows), -(-cols // BLOCK)
    scale = np.zeros((rb, cb), np.float32)
    codes = np.zeros((rows, cols), np.uint8)
    with np.errstate(all="ignore"):
        for i in range(rb):
            for j in range(cb):
                r, c = slice(i * block_rows, (i + 1) * block_rows), slice(j * BLOCK, (j + 1) * BLOCK)
                a = np.abs(x[r, c]).max()               # propagates NaN
                s = np.float32(0) if a < MIN_AMAX else np.float32(a / np.float32(448))
                inv = np.float32(0) if s == 0 else np.float32(np.float32(1) / s)
                scale[i, j] = s
                codes[r, c] = e4m3_round((x[r, c] * inv).astype(np.float32))
    return codes, scale


def values(codes: np.ndarray, scale: np.ndarray, block_rows: int) -> np.ndarray:
    """The fp64 values that codes and scales stand for."""
    rows, cols = codes.shape
    s = scale.astype(np.float64)[_block_index(rows, block_rows)][:, _block_index(cols, BLOCK)]
    with np.errstate(invalid="ignore"):
        return VALUES[codes] * s


def rmsnorm(x, weight, eps):
    """(y, rstd) in fp64."""
    x, weight = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    rstd = 1.0 / np.sqrt((x * x).mean(axis=1, keepdims=True) + eps)
    return x * rstd * weight, rstd[:, 0]


def rmsnorm_grads(dy, x, weight, eps, dh=None):
    """(dx, dweight) of sum(dy * y) + sum(dh * x) in fp64, by the chain rule
    through rstd: d rstd / d x_j = -rstd^3 x_j / n."""
    dy, x, weight = (np.asarray(t, np.float64) for t in (dy, x, weight))
    n = x.shape[1]
    rstd = rmsnorm(x, weight, eps)[1][:, None]
    d_rstd = (dy * x * weight).sum(axis=1, keepdims=True)
    dx = dy * weight * rstd - d_rstd * rstd ** 3 * x / n
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * x * rstd).sum(axis=0)
