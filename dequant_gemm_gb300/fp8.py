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

from . import (ACCUMULATE, ELEM, _call_on, _require, _require_cuda_device, _same_device, _written,
               nf4_fp8_tensor)

FP8_BLOCK = 128
FP8_DTYPE = torch.float8_e4m3fn
_F32 = torch.float32
_OUT = {torch.float32: ELEM[torch.float32], torch.bfloat16: ELEM[torch.bfloat16]}
_empty, _byref = torch.empty, ctypes.byref


@dataclass(slots=True)
class FP8Tensor:
    """codes float8_e4m3fn [rows, cols], scale float32
    [ceil(rows / block_rows), ceil(cols / 128)]; block_rows is 1 (activations,
    gradients) or 128 (weights). Plain tensors; save them with torch.save.
    Scales may have either sign; a product multiplies two of them first, which
    has to stay 0 or of magnitude 2^-126 to 2^128."""
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
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [rows, cols]")
    _check_block_rows(block_rows)
    rows, cols = x.shape
    if cols % 16:
        raise ValueError(f"cols = {cols} is not a multiple of 16")
    device = x.device
    if out is not None:
        _check_fp8(out, "out", device)
        if out.codes.shape != x.shape or out.block_rows != block_rows:
            raise ValueError(f"out holds a {out.rows}x{out.cols} tensor in blocks of "
                             f"{out.block_rows} rows, asked for {rows}x{cols} and {block_rows}")
    _require_cuda_device(device)
    q = out
    if q is None:
        q = FP8Tensor(_empty((rows, cols), dtype=FP8_DTYPE, device=device),
                      _empty((-(-rows // block_rows), -(-cols // FP8_BLOCK)), dtype=_F32, device=device),
                      block_rows)
    _call_on(device.index, "nf4_fp8_quantize", x.data_ptr(), ELEM[x.dtype], rows, cols, block_rows,
             q.codes.data_ptr(), q.scale.data_ptr())
    if out is not None:
        _written(out.codes, out.scale)
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
    _call_on(q.device.index, "nf4_fp8_dequantize", _byref(q.c_struct()), y.data_ptr(), ELEM[out_dtype])
    if out is not None:
        _written(out)
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
    # Everything that _check_matmul and the checks of `out` would refuse, in one
    # pass that does not say what it is: a small call's host time is mostly
    # such lookups.
    try:
        ac, ascale, wc, wscale = a.codes, a.scale, w.codes, w.scale
        (M, red), (rows, cols) = ac.shape, wc.shape
        device = ac.device
        row_blocks, col_blocks = (rows + 127) // FP8_BLOCK, (cols + 127) // FP8_BLOCK
        ok = (type(a) is FP8Tensor and type(w) is FP8Tensor and a.block_rows == 1
              and w.block_rows == FP8_BLOCK and red == (rows if dx else cols)
              and rows % 16 == 0 and cols % 16 == 0 and device.type == "cuda"
              and ac.dtype is FP8_DTYPE and wc.dtype is FP8_DTYPE
              and ascale.dtype is _F32 and wscale.dtype is _F32
              and ascale.shape == (M, row_blocks if dx else col_blocks)
              and wscale.shape == (row_blocks, col_blocks)
              and ac.is_contiguous() and wc.is_contiguous()
              and ascale.is_contiguous() and wscale.is_contiguous()
              and ascale.device == device and wc.device == device and wscale.device == device)
    except (AttributeError, TypeError, ValueError):
        ok = False
    if not ok:
        codes = getattr(a, "codes", None)
        device = codes.device if isinstance(codes, torch.Tensor) else None
        _check_matmul(name, a, w, dx, device)
    shape = (M, cols if dx else rows)
    if out is not None:
        if not isinstance(out, torch.Tensor):
            raise ValueError("out must be a tensor")
        out_dtype = out.dtype
    elem = _OUT.get(out_dtype)
    if elem is None:
        raise ValueError(f"the output must be float32 or bfloat16, got {out_dtype}")
    if out is not None:
        _require(out, "out", out_dtype, shape=shape)
        _same_device(device, out=out)
    elif accumulate:
        raise ValueError("accumulate=True needs the output tensor to add to (out=)")
    if not ok:
        _require_cuda_device(device)
    y = _empty(shape, dtype=out_dtype, device=device) if out is None else out
    _call_on(device.index, fn,
             _byref(nf4_fp8_tensor(ac.data_ptr(), ascale.data_ptr(), M, red, 1)),
             _byref(nf4_fp8_tensor(wc.data_ptr(), wscale.data_ptr(), rows, cols, FP8_BLOCK)),
             y.data_ptr(), elem, ACCUMULATE if accumulate else 0)
    if out is not None:
        _written(out)
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
