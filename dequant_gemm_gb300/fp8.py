"""8-bit floating point (e4m3) operands with a scale for each block of 128, and
their products.

An activation or gradient [M, K] has one fp32 scale for each 1 x 128 block, a
weight [N, K] one for each 128 x 128 block; a value is its code times its
scale. ``include/nf4gemm.h`` states the format. The weight is frozen: the
product's backward is the input gradient alone. As everywhere in the package,
the functions check their arguments, allocate outputs with PyTorch and pass
the current stream; the library's kernels do the rest.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import (ACCUMULATE, ELEM, _call_on, _check, _require, _require_cuda_device, _same_device,
               lib, nf4_fp8_tensor)

FP8_BLOCK = 128
FP8_DTYPE = torch.float8_e4m3fn


@dataclass(slots=True)
class FP8Tensor:
    """codes float8_e4m3fn [rows, cols], scale float32
    [ceil(rows / block_rows), ceil(cols / 128)]; block_rows is 1 (activations,
    gradients) or 128 (weights). Plain tensors; save them with torch.save."""
    codes: torch.Tensor
    scale: torch.Tensor
    block_rows: int = 1

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    @property
    def cols(self) -> int:
        return self.codes.shape[1]

    @property
    def device(self) -> torch.device:
        return self.codes.device

    def nbytes(self) -> int:
        return self.codes.numel() + 4 * self.scale.numel()

    def c_struct(self) -> nf4_fp8_tensor:
        rows, cols = self.codes.shape
        return nf4_fp8_tensor(self.codes.data_ptr(), self.scale.data_ptr(), rows, cols,
                              self.block_rows)


def _scale_shape(rows: int, cols: int, block_rows: int) -> tuple[int, int]:
    return -(-rows // block_rows), -(-cols // FP8_BLOCK)


def _check_block_rows(block_rows: int):
    if block_rows not in (1, FP8_BLOCK):
        raise ValueError(f"block_rows must be 1 or {FP8_BLOCK}, got {block_rows}")


def _fp8_ok(t: FP8Tensor, block_rows: int, device: torch.device) -> bool:
    """The whole check of one block-scaled tensor in one pass, without naming
    what is wrong with it (a call's host time is mostly such lookups)."""
    try:
        codes, scale = t.codes, t.scale
        rows, cols = codes.shape
        return (type(t) is FP8Tensor and t.block_rows == block_rows
                and codes.dtype is FP8_DTYPE and scale.dtype is torch.float32
                and codes.is_contiguous() and scale.is_contiguous() and cols % 16 == 0
                and scale.shape == (-(-rows // block_rows), -(-cols // FP8_BLOCK))
                and codes.device == device and scale.device == device)
    except (AttributeError, TypeError, ValueError):
        return False


def _check_fp8(t: FP8Tensor, name: str, device: torch.device):
    """Types, exact sizes, contiguity and device of one block-scaled tensor."""
    if not isinstance(t, FP8Tensor):
        raise ValueError(f"{name} must be an FP8Tensor, got {type(t)}")
    _check_block_rows(t.block_rows)
    _require(t.codes, f"{name}.codes", FP8_DTYPE)
    if t.codes.dim() != 2:
        raise ValueError(f"{name}.codes must be 2-D [rows, cols]")
    rows, cols = t.codes.shape
    if cols % 16:
        raise ValueError(f"{name}: cols = {cols} is not a multiple of 16")
    _require(t.scale, f"{name}.scale", torch.float32, shape=_scale_shape(rows, cols, t.block_rows))
    _same_device(device, **{f"{name}.codes": t.codes, f"{name}.scale": t.scale})


def alloc_fp8(rows: int, cols: int, device, block_rows: int = 1) -> FP8Tensor:
    _check_block_rows(block_rows)
    return FP8Tensor(torch.empty((rows, cols), dtype=FP8_DTYPE, device=device),
                     torch.empty(_scale_shape(rows, cols, block_rows), dtype=torch.float32,
                                 device=device), block_rows)


def nf4_fp8_quantize(x: torch.Tensor, block_rows: int = 1,
                     out: FP8Tensor | None = None) -> FP8Tensor:
    """Quantize an fp32, bf16 or fp16 [rows, cols] CUDA tensor (cols a multiple
    of 16) in 1 x 128 blocks (activations, gradients) or, with block_rows 128,
    in 128 x 128 blocks (weights)."""
    if not isinstance(x, torch.Tensor) or x.dtype not in ELEM:
        raise ValueError(f"x must be float32, bfloat16 or float16, got {getattr(x, 'dtype', type(x))}")
    _require(x, "x", x.dtype)
    if x.dim() != 2:
        raise ValueError("x must be 2-D [rows, cols]")
    _check_block_rows(block_rows)
    rows, cols = x.shape
    if cols % 16:
        raise ValueError(f"cols = {cols} is not a multiple of 16")
    if out is not None:
        _check_fp8(out, "out", x.device)
        if out.codes.shape != x.shape or out.block_rows != block_rows:
            raise ValueError(f"out holds a {out.rows}x{out.cols} tensor in blocks of "
                             f"{out.block_rows} rows, asked for {rows}x{cols} and {block_rows}")
    _require_cuda_device(x.device)
    q = out if out is not None else alloc_fp8(rows, cols, x.device, block_rows)
    _check("nf4_fp8_quantize",
           _call_on(x.device, lib().nf4_fp8_quantize, x.data_ptr(), ELEM[x.dtype], rows, cols,
                    block_rows, q.codes.data_ptr(), q.scale.data_ptr()))
    return q


def nf4_fp8_dequantize(q: FP8Tensor, out: torch.Tensor | None = None,
                       out_dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """[rows, cols] values of q in fp32, or rounded to bf16 or fp16 (for checks
    and export)."""
    _check_fp8(q, "q", q.device if isinstance(q, FP8Tensor) else None)
    if out is not None:
        if not isinstance(out, torch.Tensor):
            raise ValueError("out must be a tensor")
        out_dtype = out.dtype
    if out_dtype not in ELEM:
        raise ValueError(f"the output must be float32, bfloat16 or float16, got {out_dtype}")
    if out is not None:
        _require(out, "out", out_dtype, shape=q.codes.shape)
        _same_device(q.device, out=out)
    _require_cuda_device(q.device)
    y = out if out is not None else torch.empty(q.codes.shape, dtype=out_dtype, device=q.device)
    _check("nf4_fp8_dequantize",
           _call_on(q.device, lib().nf4_fp8_dequantize, ctypes.byref(q.c_struct()), y.data_ptr(),
                    ELEM[out_dtype]))
    return y


def _check_matmul(name: str, a: FP8Tensor, w: FP8Tensor, dx: bool, device):
    """Raises for what is wrong with a product's operands, if anything is."""
    _check_fp8(a, name, device)
    _check_fp8(w, "weight", device)
    if a.block_rows != 1 or w.block_rows != FP8_BLOCK:
        raise ValueError(f"{name} must have block_rows 1 and the weight {FP8_BLOCK}, got "
                         f"{a.block_rows} and {w.block_rows}")
    if w.rows % 16:
        raise ValueError(f"weight: rows = {w.rows} is not a multiple of 16")
    want = w.rows if dx else w.cols
    if a.cols != want:
        raise ValueError(f"{name} must be [M, {want}], got [{a.rows}, {a.cols}]")


def _matmul(name: str, fn: str, a: FP8Tensor, w: FP8Tensor, dx: bool, out, out_dtype,
            accumulate: bool) -> torch.Tensor:
    codes = getattr(a, "codes", None)
    device = codes.device if isinstance(codes, torch.Tensor) else None
    if not (_fp8_ok(a, 1, device) and _fp8_ok(w, FP8_BLOCK, device)):
        _check_matmul(name, a, w, dx, device)
    M, red = codes.shape
    rows, cols = w.codes.shape
    if rows % 16 or red != (rows if dx else cols):
        _check_matmul(name, a, w, dx, device)
    shape = (M, cols if dx else rows)
    if out is not None:
        if not isinstance(out, torch.Tensor):
            raise ValueError("out must be a tensor")
        out_dtype = out.dtype
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"the output must be float32 or bfloat16, got {out_dtype}")
    if out is not None:
        _require(out, "out", out_dtype, shape=shape)
        _same_device(device, out=out)
    elif accumulate:
        raise ValueError("accumulate=True needs the output tensor to add to (out=)")
    _require_cuda_device(device)
    y = out if out is not None else torch.empty(shape, dtype=out_dtype, device=device)
    _check(fn, _call_on(
        device, getattr(lib(), fn),
        ctypes.byref(nf4_fp8_tensor(codes.data_ptr(), a.scale.data_ptr(), M, red, 1)),
        ctypes.byref(nf4_fp8_tensor(w.codes.data_ptr(), w.scale.data_ptr(), rows, cols, FP8_BLOCK)),
        y.data_ptr(), ELEM[out_dtype], ACCUMULATE if accumulate else 0))
    return y


def nf4_fp8_matmul_fwd(X: FP8Tensor, w: FP8Tensor, out: torch.Tensor | None = None,
                       out_dtype: torch.dtype = torch.float32,
                       accumulate: bool = False) -> torch.Tensor:
    """Y = value(X) * value(w)^T (+ out when accumulate): X [M, cols] with
    1 x 128 blocks, w [rows, cols] with 128 x 128 blocks -> Y fp32 or bf16
    [M, rows]. rows and cols are multiples of 16."""
    return _matmul("X", "nf4_fp8_matmul_fwd", X, w, False, out, out_dtype, accumulate)


def nf4_fp8_matmul_bwd_dx(dY: FP8Tensor, w: FP8Tensor, out: torch.Tensor | None = None,
                          out_dtype: torch.dtype = torch.float32,
                          accumulate: bool = False) -> torch.Tensor:
    """dX = value(dY) * value(w) (+ out when accumulate): dY [M, rows] with
    1 x 128 blocks along rows -> dX fp32 or bf16 [M, cols]. No dW."""
    return _matmul("dY", "nf4_fp8_matmul_bwd_dx", dY, w, True, out, out_dtype, accumulate)
