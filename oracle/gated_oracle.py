"""Plain CPU oracle of the gated block's activations and of the 4-bit weights in
groups: the definitions written down in numpy, sharing no code with the CUDA
library. TEST INFRASTRUCTURE ONLY.

Activations are fp64, by their own formulas (SiLU by the logistic function, the
tanh form of GELU by tanh). The 4-bit format fixes its steps to fp32, which
numpy float32 takes with one IEEE rounding each.
"""
from __future__ import annotations

import numpy as np

_ROOT = np.sqrt(2.0 / np.pi)


def act(g, name: str):
    """(act(g), act'(g))."""
    g = np.asarray(g, np.float64)
    if name == "silu":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    t = np.tanh(_ROOT * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * _ROOT * (1.0 + 3 * 0.044715 * g * g)


def exponent(g, name: str):
    """p(g) of act(g) = g sigma(p(g)), and p'(g)."""
    g = np.asarray(g, np.float64)
    c0, c1 = (1.0, 0.0) if name == "silu" else (2 * _ROOT, 2 * _ROOT * 0.044715)
    return g * (c0 + c1 * g * g), c0 + 3 * c1 * g * g


def _bf16(x: np.ndarray) -> np.ndarray:
    """fp32 rounded to bf16 (nearest even), as fp32; finite values."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7fff + ((b >> 16) & 1)) & 0xffff0000
    return b.astype(np.uint32).view(np.float32)


def int4_quantize(w, group: int, zero_point: bool, scale: str):
    """(codes uint8 [rows, cols], scale float32 [rows, groups], zero) of fp32
    values; scale "bf16" or "f16" is the type that the scales are rounded to."""
    w = np.asarray(w, np.float32)
    rows, cols = w.shape
    g = w.reshape(rows, cols // group, group)
    if zero_point:
        lo, hi = np.minimum(g.min(2), np.float32(0)), np.maximum(g.max(2), np.float32(0))
        raw = (hi - lo) / np.float32(15)
    else:
        raw = np.abs(g).max(2) / np.float32(7)
    s = _bf16(raw) if scale == "bf16" else raw.astype(np.float16).astype(np.float32)
    live = np.where(s == 0, np.float32(1), s)
    if zero_point:
        z = np.where(s == 0, np.float32(0), np.clip(np.rint(-lo / live), 0, 15))
    else:
        z = np.full_like(s, 8)
    q = np.clip(np.rint(g / live[:, :, None]) + z[:, :, None], 0, 15)
    q = np.where((s == 0)[:, :, None], z[:, :, None], q)
    return q.reshape(rows, cols).astype(np.uint8), s, z.astype(np.uint8)


def int4_pack(q: np.ndarray) -> np.ndarray:
    """The even element of a pair in the high half of its byte."""
    return (q[:, 0::2] << 4 | q[:, 1::2]).astype(np.uint8)


def int4_values(codes: np.ndarray, scale, zero) -> np.ndarray:
    """fp64 values of packed codes, scales and zero points (None: 8)."""
    rows, half = codes.shape
    q = np.empty((rows, 2 * half), np.int64)
    q[:, 0::2], q[:, 1::2] = codes >> 4, codes & 15
    group = 2 * half // scale.shape[1]
    z = 8 if zero is None else np.repeat(zero.astype(np.int64), group, 1)
    return (q - z) * np.repeat(np.asarray(scale, np.float64), group, 1)
