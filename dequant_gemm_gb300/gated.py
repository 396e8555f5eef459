"""The gated feed-forward block on 8-bit operands: both projections, the
activation and the product in one kernel, and its gradients.

    G = X gate^T,  U = X up^T,  Y = act(G) * U,  act(g) = g sigma(p(g))

with p(g) = g for "silu" and 2 sqrt(2 / pi) (g + 0.044715 g^3) for "gelu_tanh".
Y leaves in 8 bits, as the next product reads it, or in 16 or 32. The weights
are frozen: the backward is the input gradient alone, from the G and U that
the forward keeps in bf16.
"""
from __future__ import annotations

import ctypes
import sys
from array import array

import torch

from . import (ACCUMULATE, ELEM, NF4Error, _call_on, _require, _require_cuda_device, _same_device,
               _written, nf4_fp8_tensor)
from .fp8 import FP8_BLOCK, FP8_DTYPE, FP8Tensor, _check_fp8, _check_matmul, _empty, _F32, _OUT
from .norm import _refused, _require_matrix

ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}
_BF16 = torch.bfloat16


def _activation(name: str) -> int:
    code = ACTIVATIONS.get(name) if isinstance(name, str) else None
    if code is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {name!r}")
    return code


# Two to four nf4_fp8_tensor in a row, built at once: five 64-bit words each (the
# low half of the last is block_rows), whose addresses the calls take. One ctypes
# struct after the other took the host 0.6 us each.
_STRUCT = ctypes.sizeof(nf4_fp8_tensor)
assert _STRUCT == 8 * 5 and array("q").itemsize == 8 and sys.byteorder == "little"


def _plain_pair(gate, up):
    """(rows, cols, device, words of both structs) of a pair that passes _check_pair,
    in one pass; None where it does not."""
    try:
        gc, gs, uc, us = gate.codes, gate.scale, up.codes, up.scale
        rows, cols = shape = gc.shape
        device = gc.device
        blocks = ((rows + 127) // FP8_BLOCK, (cols + 127) // FP8_BLOCK)
        if (type(gate) is FP8Tensor and type(up) is FP8Tensor and gate.block_rows == FP8_BLOCK
                and up.block_rows == FP8_BLOCK and rows % 16 == 0 and cols % 16 == 0
                and gc.dtype is FP8_DTYPE and uc.dtype is FP8_DTYPE and uc.shape == shape
                and gs.dtype is _F32 and us.dtype is _F32 and gs.shape == blocks and us.shape == blocks
                and gc.is_contiguous() and uc.is_contiguous() and gs.is_contiguous() and us.is_contiguous()
                and gs.device == device and uc.device == device and us.device == device):
            return rows, cols, device, (gc.data_ptr(), gs.data_ptr(), rows, cols, FP8_BLOCK,
                                        uc.data_ptr(), us.data_ptr(), rows, cols, FP8_BLOCK)
    except (AttributeError, TypeError, ValueError):
        pass
    return None


def _plain_left(a, cols, device):
    """The words of an operand [M, cols] with 1 x 128 blocks, or None."""
    try:
        codes, scale = a.codes, a.scale
        m, k = codes.shape
        if (type(a) is FP8Tensor and a.block_rows == 1 and k == cols and codes.dtype is FP8_DTYPE
                and scale.dtype is _F32 and scale.shape == (m, (cols + 127) // FP8_BLOCK)
                and codes.is_contiguous() and scale.is_contiguous() and codes.device == device
                and scale.device == device):
            return codes.data_ptr(), scale.data_ptr(), m, cols, 1
    except (AttributeError, TypeError, ValueError):
        pass
    return None


def _device_of(t):
    codes = getattr(t, "codes", None)
    return codes.device if isinstance(codes, torch.Tensor) else None


def _check_pair(name: str, a, gate, up, dx: bool):
    """Raises for what is wrong with a left operand and the two weights, if anything is."""
    device = _device_of(a)
    _check_fp8(a, name, device)
    for w, which in ((gate, "gate"), (up, "up")):
        _check_fp8(w, which, device)
        if w.block_rows != FP8_BLOCK:
            raise ValueError(f"{which} must have block_rows {FP8_BLOCK}, got {w.block_rows}")
    if gate.codes.shape != up.codes.shape:
        raise ValueError(f"gate and up must have the same shape, got {tuple(gate.codes.shape)} and "
                         f"{tuple(up.codes.shape)}")
    _check_matmul(name, a, gate, dx, device)


def _words(t: FP8Tensor):
    rows, cols = t.codes.shape
    return t.codes.data_ptr(), t.scale.data_ptr(), rows, cols, t.block_rows


def nf4_fp8_gated_fwd(X: FP8Tensor, gate: FP8Tensor, up: FP8Tensor, activation: str = "silu",
                      out_dtype: torch.dtype = FP8_DTYPE, save: bool = False):
    """Y = act(value(X) value(gate)^T) * (value(X) value(up)^T): X [M, cols] with
    1 x 128 blocks, gate and up [rows, cols] with 128 x 128 blocks (rows and cols
    multiples of 16). Returns (y, g, u).

    out_dtype: torch.float8_e4m3fn makes y an FP8Tensor in 1 x 128 blocks, which
    the down product reads; float32 or bfloat16 a [M, rows] tensor. g and u are
    the two projections in bf16 (what nf4_fp8_gated_bwd reads), None unless
    save. Y is taken from the fp32 projections and rounded once."""
    pair = _plain_pair(gate, up)
    left = None if pair is None else _plain_left(X, pair[1], pair[2])
    if left is None:
        _check_pair("X", X, gate, up, False)
        left, pair = _words(X), (gate.rows, gate.cols, X.device, _words(gate) + _words(up))
    rows, _, device, words = pair
    act = _activation(activation)
    fp8 = out_dtype == FP8_DTYPE
    if not fp8 and out_dtype not in _OUT:
        raise ValueError(f"the output must be float8_e4m3fn, float32 or bfloat16, got {out_dtype}")
    _require_cuda_device(device)
    M = left[2]
    if fp8:
        codes = _empty((M, rows), dtype=FP8_DTYPE, device=device)
        scale = _empty((M, (rows + 127) // FP8_BLOCK), dtype=_F32, device=device)
        y, y_ptr, elem, scale_ptr = FP8Tensor(codes, scale), codes.data_ptr(), 0, scale.data_ptr()
    else:
        y = _empty((M, rows), dtype=out_dtype, device=device)
        y_ptr, elem, scale_ptr = y.data_ptr(), _OUT[out_dtype], None
    g = u = None
    if save:
        g, u = (_empty((M, rows), dtype=_BF16, device=device) for _ in range(2))
    structs = array("q", left + words)
    at = structs.buffer_info()[0]
    _call_on(device.index, "nf4_fp8_gated_fwd", at, at + _STRUCT, at + 2 * _STRUCT, act, y_ptr, elem,
             scale_ptr, None if g is None else g.data_ptr(), None if u is None else u.data_ptr())
    return y, g, u


def _check_bwd(dy, g, u):
    """Raises for what is wrong with the operands of nf4_fp8_gated_bwd."""
    _require_matrix(dy, "dy")
    if dy.dim() != 2:
        raise ValueError(f"dy must be 2-D [M, rows], got {tuple(dy.shape)}")
    for t, name in ((g, "g"), (u, "u")):
        _require(t, name, _BF16, shape=dy.shape)
        _same_device(dy.device, **{name: t})
    if dy.shape[1] % 16:
        raise ValueError(f"rows = {dy.shape[1]} is not a multiple of 16")


def nf4_fp8_gated_bwd(dy: torch.Tensor, g: torch.Tensor, u: torch.Tensor, activation: str = "silu"):
    """(dG, dU) from the gradient of Y: dG = dy u act'(g), dU = dy act(g), taken in
    fp32 and quantized in 1 x 128 blocks. dy [M, rows] is fp32, bf16 or fp16, g
    and u are bf16 as nf4_fp8_gated_fwd kept them; rows a multiple of 16. Every
    tensor is contiguous and starts on a 16-byte boundary."""
    try:
        M, rows = shape = dy.shape
        device = dy.device
        ok = (dy.dtype in ELEM and g.dtype is _BF16 and u.dtype is _BF16 and g.shape == shape and u.shape == shape
              and rows % 16 == 0 and dy.is_contiguous() and g.is_contiguous() and u.is_contiguous()
              and g.device == device and u.device == device)
    except (AttributeError, TypeError, ValueError):
        ok = False
    if not ok:
        _check_bwd(dy, g, u)
    act = _activation(activation)
    _require_cuda_device(device)
    nb = (rows + 127) // FP8_BLOCK
    dg, du = (FP8Tensor(_empty((M, rows), dtype=FP8_DTYPE, device=device),
                        _empty((M, nb), dtype=_F32, device=device)) for _ in range(2))
    try:
        _call_on(device.index, "nf4_fp8_gated_bwd", dy.data_ptr(), ELEM[dy.dtype], g.data_ptr(), u.data_ptr(), M,
                 rows, act, dg.codes.data_ptr(), dg.scale.data_ptr(), du.codes.data_ptr(), du.scale.data_ptr())
    except NF4Error as error:
        _refused(error, dy=dy, g=g, u=u)
    return dg, du


def nf4_fp8_gated_bwd_dx(dG: FP8Tensor, dU: FP8Tensor, gate: FP8Tensor, up: FP8Tensor,
                         out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32,
                         accumulate: bool = False) -> torch.Tensor:
    """dX = value(dG) value(gate) + value(dU) value(up) (+ out when accumulate):
    dG, dU [M, rows] with 1 x 128 blocks -> dX fp32 or bf16 [M, cols], one sum
    over both weights. No dW."""
    pair = _plain_pair(gate, up)
    left = right = None
    if pair is not None:
        left, right = _plain_left(dG, pair[0], pair[2]), _plain_left(dU, pair[0], pair[2])
    if left is None or right is None or left[2] != right[2]:
        _check_pair("dG", dG, gate, up, True)
        _check_matmul("dU", dU, up, True, dG.device)
        if dU.rows != dG.rows:
            raise ValueError(f"dG and dU must have the same rows, got {dG.rows} and {dU.rows}")
        left, right = _words(dG), _words(dU)
        pair = (gate.rows, gate.cols, dG.device, _words(gate) + _words(up))
    M, (_, cols, device, words) = left[2], pair
    if out is not None:
        if not isinstance(out, torch.Tensor):
            raise ValueError("out must be a tensor")
        out_dtype = out.dtype
    elem = _OUT.get(out_dtype)
    if elem is None:
        raise ValueError(f"the output must be float32 or bfloat16, got {out_dtype}")
    if out is not None:
        _require(out, "out", out_dtype, shape=(M, cols))
        _same_device(device, out=out)
    elif accumulate:
        raise ValueError("accumulate=True needs the output tensor to add to (out=)")
    _require_cuda_device(device)
    dx = _empty((M, cols), dtype=out_dtype, device=device) if out is None else out
    structs = array("q", left + right + words)
    at = structs.buffer_info()[0]
    _call_on(device.index, "nf4_fp8_gated_bwd_dx", at, at + _STRUCT, at + 2 * _STRUCT, at + 3 * _STRUCT,
             dx.data_ptr(), elem, ACCUMULATE if accumulate else 0)
    if out is not None:
        _written(out)
    return dx
