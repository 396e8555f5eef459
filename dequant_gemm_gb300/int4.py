"""Uniform 4-bit weights with a 16-bit scale, and a zero point, for each group of
32, 64 or 128 values along a row, and products of few tokens with them, for
decoding.

A value is (code - zero point) * scale; ``include/nf4gemm.h`` states the
format: two codes a byte in the order of the row, scales and zero points not
packed. Checkpoints that hold such weights otherwise (eight codes an int32,
transposed or interleaved columns, packed or shifted zero points) have to be
brought into this order first; nothing here does. As everywhere in the package, the functions check their arguments,
allocate outputs with PyTorch and pass the current stream.
"""
from __future__ import annotations

import ctypes
from array import array
from dataclasses import dataclass

import torch

from . import (ACCUMULATE, ELEM, NF4Error, _call_on, _require, _require_cuda_device, _same_device,
               _written, nf4_int4_weight)
from .gated import _activation
from .norm import _refused, _require_matrix

INT4_GROUPS = (32, 64, 128)
INT4_MAX_COLS = 262144         # NF4_INT4_MAX_COLS
_SCALES = {torch.bfloat16: ELEM[torch.bfloat16], torch.float16: ELEM[torch.float16]}
_U8, _empty = torch.uint8, torch.empty

# An nf4_int4_weight as six 64-bit words (little-endian: the group, and the scales'
# type above it), whose address the calls take: as a ctypes struct it took the host
# 1 us more.
_STRUCT = ctypes.sizeof(nf4_int4_weight)
assert _STRUCT == 8 * 6


@dataclass(slots=True)
class Int4Weight:
    """codes uint8 [rows, cols / 2] (element 2j of a row in the high half of byte
    j), scale float16 or bfloat16 [rows, cols / group], zero uint8 [rows,
    cols / group] (0 to 15) or None, which means 8 everywhere. Plain tensors;
    save them with torch.save."""
    codes: torch.Tensor
    scale: torch.Tensor
    zero: torch.Tensor | None = None

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    @property
    def cols(self) -> int:
        return 2 * self.codes.shape[1]

    @property
    def group(self) -> int:
        """Values of a row that share a scale (128 where there are none)."""
        return self.cols // self.scale.shape[1] if self.scale.shape[1] else 128

    @property
    def device(self) -> torch.device:
        return self.codes.device

    def nbytes(self) -> int:
        n = self.codes.numel() + 2 * self.scale.numel()
        return n + (0 if self.zero is None else self.zero.numel())

    def words(self) -> tuple:
        """The fields of the C struct, a word each."""
        return (self.codes.data_ptr(), self.scale.data_ptr(), 0 if self.zero is None else self.zero.data_ptr(),
                self.rows, self.cols, self.group | _SCALES[self.scale.dtype] << 32)


def _check_group(group: int):
    if group not in INT4_GROUPS:
        raise ValueError(f"group must be one of {INT4_GROUPS}, got {group}")


def _check_int4(w: Int4Weight, name: str, device):
    """Types, exact sizes, contiguity and device of one 4-bit weight."""
    if not isinstance(w, Int4Weight):
        raise ValueError(f"{name} must be an Int4Weight, got {type(w)}")
    _require(w.codes, f"{name}.codes", _U8)
    if not isinstance(w.scale, torch.Tensor) or w.scale.dtype not in _SCALES:
        raise ValueError(f"{name}.scale must be float16 or bfloat16, got {getattr(w.scale, 'dtype', type(w.scale))}")
    if w.codes.dim() != 2 or w.scale.dim() != 2:
        raise ValueError(f"{name}.codes and {name}.scale must be 2-D [rows, cols / 2] and [rows, cols / group]")
    rows, cols, groups = w.rows, w.cols, w.scale.shape[1]
    if (cols % groups if groups else cols):
        raise ValueError(f"{name}: {cols} columns in {groups} groups")
    _check_group(w.group)
    _require(w.scale, f"{name}.scale", w.scale.dtype, shape=(rows, groups))
    _same_device(device, **{f"{name}.codes": w.codes, f"{name}.scale": w.scale})
    if w.zero is not None:
        _require(w.zero, f"{name}.zero", _U8, shape=(rows, groups))
        _same_device(device, **{f"{name}.zero": w.zero})


def _plain_int4(w, device):
    """The words of a weight that passes _check_int4, in one pass; None where it
    does not."""
    try:
        codes, scale, zero = w.codes, w.scale, w.zero
        rows, half = codes.shape
        groups = scale.shape[1]
        group = 2 * half // groups
        if (type(w) is Int4Weight and codes.dtype is _U8 and scale.dtype in _SCALES and group in INT4_GROUPS
                and group * groups == 2 * half and scale.shape == (rows, groups) and codes.is_contiguous()
                and scale.is_contiguous() and codes.device == device and scale.device == device
                and (zero is None or zero.dtype is _U8 and zero.shape == scale.shape and zero.is_contiguous()
                     and zero.device == device)):
            return (codes.data_ptr(), scale.data_ptr(), 0 if zero is None else zero.data_ptr(), rows, 2 * half,
                    group | _SCALES[scale.dtype] << 32)
    except (AttributeError, TypeError, ValueError, IndexError, ZeroDivisionError):
        pass
    return None


def nf4_int4_quantize(W: torch.Tensor, group: int = 128, zero_point: bool = True,
                      scale_dtype: torch.dtype = torch.bfloat16, out: Int4Weight | None = None) -> Int4Weight:
    """Quantize a finite fp32, bf16 or fp16 [rows, cols] CUDA tensor (cols a
    multiple of group) to nearest: with a zero point for each group over the
    range of its values and 0, or symmetrically about code 8."""
    _require_matrix(W, "W")
    if W.dim() != 2:
        raise ValueError("W must be 2-D [rows, cols]")
    _check_group(group)
    if scale_dtype not in _SCALES:
        raise ValueError(f"scale_dtype must be float16 or bfloat16, got {scale_dtype}")
    rows, cols = W.shape
    if cols % group:
        raise ValueError(f"cols = {cols} is not a multiple of the group, {group}")
    device = W.device
    if out is not None:
        _check_int4(out, "out", device)
        if (out.codes.shape != (rows, cols // 2) or out.scale.shape[1] != cols // group
                or out.scale.dtype != scale_dtype or (out.zero is not None) != zero_point):
            raise ValueError(f"out is a {out.rows}x{out.cols} weight in groups of {out.group} with {out.scale.dtype} "
                             f"scales and {'no ' if out.zero is None else ''}zero points; asked for {rows}x{cols}, "
                             f"{group}, {scale_dtype} and zero_point={zero_point}")
    _require_cuda_device(device)
    q = out
    if q is None:
        shape = (rows, cols // group)
        q = Int4Weight(_empty((rows, cols // 2), dtype=_U8, device=device),
                       _empty(shape, dtype=scale_dtype, device=device),
                       _empty(shape, dtype=_U8, device=device) if zero_point else None)
    try:
        _call_on(device.index, "nf4_int4_quantize", W.data_ptr(), ELEM[W.dtype], rows, cols, group,
                 _SCALES[scale_dtype], q.codes.data_ptr(), q.scale.data_ptr(),
                 None if q.zero is None else q.zero.data_ptr())
    except NF4Error as error:
        _refused(error, W=W, **{"out.codes": q.codes})
    if out is not None:
        _written(out.codes, out.scale, out.zero)
    return q


def nf4_int4_dequantize(w: Int4Weight, out: torch.Tensor | None = None,
                        out_dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """[rows, cols] values of w in fp32, or rounded to bf16 or fp16 (for export and
    for library products of many tokens)."""
    _check_int4(w, "w", w.device if isinstance(w, Int4Weight) and isinstance(w.codes, torch.Tensor) else None)
    if out is not None:
        if not isinstance(out, torch.Tensor):
            raise ValueError("out must be a tensor")
        out_dtype = out.dtype
    if out_dtype not in ELEM:
        raise ValueError(f"the output must be float32, bfloat16 or float16, got {out_dtype}")
    shape = (w.rows, w.cols)
    if out is not None:
        _require(out, "out", out_dtype, shape=shape)
        _same_device(w.device, out=out)
    _require_cuda_device(w.device)
    y = out if out is not None else _empty(shape, dtype=out_dtype, device=w.device)
    try:
        struct = array("q", w.words())
        _call_on(w.device.index, "nf4_int4_dequantize", struct.buffer_info()[0], y.data_ptr(), ELEM[out_dtype])
    except NF4Error as error:
        _refused(error, out=out, **{"w.codes": w.codes})
    if out is not None:
        _written(out)
    return y


def _check_x(X, **weights):
    """Raises for what is wrong with the activations and the weights of a product,
    if anything is."""
    if not isinstance(X, torch.Tensor) or X.dtype not in _SCALES:
        raise ValueError(f"X must be bfloat16 or float16, got {getattr(X, 'dtype', type(X))}")
    _require(X, "X", X.dtype)
    for name, w in weights.items():
        _check_int4(w, name, X.device)
        if w.cols > INT4_MAX_COLS:
            raise ValueError(f"{name}: {w.cols} columns; products take {INT4_MAX_COLS} at most (dequantize longer rows)")
        if X.dim() != 2 or X.shape[1] != w.cols:
            raise ValueError(f"X must be [M, {w.cols}]")


def _plain_x(X) -> bool:
    return (isinstance(X, torch.Tensor) and X.dtype in _SCALES and X.dim() == 2 and X.is_contiguous()
            and X.device.type == "cuda")


def nf4_int4_matmul_fwd(X: torch.Tensor, w: Int4Weight, out: torch.Tensor | None = None,
                        out_dtype: torch.dtype = torch.float32, accumulate: bool = False) -> torch.Tensor:
    """Y = X * value(w)^T (+ out when accumulate): X bf16 or fp16 [M, cols] -> Y
    fp32, bf16 or fp16 [M, rows]. For few tokens: the weight is read once for
    every 16."""
    words = _plain_int4(w, X.device) if _plain_x(X) else None
    if words is None or X.shape[1] != words[4] or words[4] > INT4_MAX_COLS:
        _check_x(X, w=w)
        words = w.words()
    M, rows = X.shape[0], words[3]
    if out is not None:
        if not isinstance(out, torch.Tensor):
            raise ValueError("out must be a tensor")
        out_dtype = out.dtype
    elem = ELEM.get(out_dtype)
    if elem is None:
        raise ValueError(f"the output must be float32, bfloat16 or float16, got {out_dtype}")
    if out is not None:
        _require(out, "out", out_dtype, shape=(M, rows))
        _same_device(X.device, out=out)
    elif accumulate:
        raise ValueError("accumulate=True needs the output tensor to add to (out=)")
    device = X.device
    _require_cuda_device(device)
    y = _empty((M, rows), dtype=out_dtype, device=device) if out is None else out
    try:
        struct = array("q", words)
        _call_on(device.index, "nf4_int4_matmul_fwd", X.data_ptr(), _SCALES[X.dtype], M, struct.buffer_info()[0],
                 y.data_ptr(), elem, ACCUMULATE if accumulate else 0)
    except NF4Error as error:
        _refused(error, X=X, **{"w.codes": w.codes})
    if out is not None:
        _written(out)
    return y


def nf4_int4_gated_fwd(X: torch.Tensor, gate: Int4Weight, up: Int4Weight, activation: str = "silu",
                       out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """The gated block for few tokens, in one kernel: act(X value(gate)^T) *
    (X value(up)^T), X bf16 or fp16 [M, cols] -> fp32, bf16 or fp16 [M, rows]
    (default: X's type). gate and up have the same shape, group and scale type,
    each with or without zero points."""
    a = b = None
    if _plain_x(X):
        a, b = _plain_int4(gate, X.device), _plain_int4(up, X.device)
    if a is None or b is None or X.shape[1] != a[4] or a[4] > INT4_MAX_COLS:
        _check_x(X, gate=gate)
        _check_int4(up, "up", X.device)
        a, b = gate.words(), up.words()
    if a[3:] != b[3:]:
        raise ValueError("gate and up must have the same shape, group and scale type")
    act = _activation(activation)
    out_dtype = X.dtype if out_dtype is None else out_dtype
    elem = ELEM.get(out_dtype)
    if elem is None:
        raise ValueError(f"the output must be float32, bfloat16 or float16, got {out_dtype}")
    device = X.device
    _require_cuda_device(device)
    M = X.shape[0]
    y = _empty((M, a[3]), dtype=out_dtype, device=device)
    try:
        structs = array("q", a + b)
        at = structs.buffer_info()[0]
        _call_on(device.index, "nf4_int4_gated_fwd", X.data_ptr(), _SCALES[X.dtype], M, at, at + _STRUCT, act,
                 y.data_ptr(), elem)
    except NF4Error as error:
        _refused(error, X=X, **{"gate.codes": gate.codes, "up.codes": up.codes})
    return y
