"""RMS norm with the residual's addition, writing 8-bit operands for the fp8
products or 16/32-bit values, and its gradients."""
from __future__ import annotations

import torch

from . import (ELEM, NF4Error, _call_on, _require, _require_cuda_device, _same_device,
               _written, lib)
from .fp8 import FP8_BLOCK, FP8_DTYPE, FP8Tensor


_F32, _empty = torch.float32, torch.empty


def _require_matrix(t, name: str, shape=None):
    if not isinstance(t, torch.Tensor) or t.dtype not in ELEM:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {getattr(t, 'dtype', type(t))}")
    _require(t, name, t.dtype, shape=shape)


def _check_norm(x, name: str, weight):
    _require_matrix(x, name)
    if x.dim() != 2 or x.shape[1] == 0:
        raise ValueError(f"{name} must be 2-D [rows, cols] with cols > 0, got {tuple(x.shape)}")
    _require_matrix(weight, "weight", (x.shape[1],))
    if weight.device != x.device:
        _same_device(x.device, weight=weight)


def _plain_matrix(x, weight) -> bool:
    """Whether x [rows, cols] and weight [cols] pass _check_norm, in one pass
    that does not say why not."""
    try:
        rows, cols = x.shape
        return (x.dtype in ELEM and weight.dtype in ELEM and weight.shape == (cols,) and cols > 0
                and x.is_contiguous() and weight.is_contiguous() and weight.device == x.device)
    except (AttributeError, TypeError, ValueError):
        return False


def _check_fwd(x, weight, residual):
    """Raises for what is wrong with the forward's inputs, if anything is."""
    _check_norm(x, "x", weight)
    if residual is not None:
        _require_matrix(residual, "residual", x.shape)
        if residual.dtype not in (x.dtype, torch.float32):
            raise ValueError(f"residual must be {x.dtype} or float32, got {residual.dtype}")
        _same_device(x.device, residual=residual)


def _like(t, h) -> bool:
    """Whether t has h's type, shape and device and is contiguous."""
    return (isinstance(t, torch.Tensor) and t.dtype is h.dtype and t.shape == h.shape
            and t.is_contiguous() and t.device == h.device)


def _refused(error: NF4Error, **tensors):
    """Raises ValueError with the name of the operand that a call was refused for
    where that is its alignment, else the call's own error."""
    for name, t in tensors.items():
        if error.status == 3 and t is not None and t.data_ptr() % 16:
            raise ValueError(f"{name} must start on a 16-byte boundary (a row slice of an odd width "
                             f"need not: clone it)") from error
    raise error


def nf4_rmsnorm_fwd(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                    eps: float = 1e-6, out_dtype: torch.dtype | None = None,
                    save_rstd: bool = False, out_h: torch.Tensor | None = None):
    """h = x + residual (rounded to the residual's type; h = x without one) and
    y = h / sqrt(mean(h^2) + eps) * weight, per row. Returns (y, h, rstd).

    x [rows, cols] and weight [cols] are fp32, bf16 or fp16; the residual is of
    x's type or fp32. out_dtype: fp32, bf16, fp16 (default: x's type), or
    torch.float8_e4m3fn, which makes y an FP8Tensor in 1 x 128 blocks (cols a
    multiple of 16). rstd (fp32 [rows]) is what the backward needs, None
    unless save_rstd. out_h: where to write h; the residual itself may be
    given, to update the stream in place. Every tensor is contiguous and starts
    on a 16-byte boundary, which a row slice of an odd width need not."""
    if not _plain_matrix(x, weight) or residual is not None and not (
            isinstance(residual, torch.Tensor) and residual.shape == x.shape
            and (residual.dtype is x.dtype or residual.dtype is torch.float32)
            and residual.is_contiguous() and residual.device == x.device):
        _check_fwd(x, weight, residual)
    rows, cols = x.shape
    if out_h is not None:
        if residual is None:
            raise ValueError("out_h without a residual: h is x itself")
        _require(out_h, "out_h", residual.dtype, shape=x.shape)
        _same_device(x.device, out_h=out_h)
    out_dtype = x.dtype if out_dtype is None else out_dtype
    fp8 = out_dtype == FP8_DTYPE
    if not fp8 and out_dtype not in ELEM:
        raise ValueError(f"the output must be float32, bfloat16, float16 or float8_e4m3fn, got {out_dtype}")
    if fp8 and cols % 16:
        raise ValueError(f"cols = {cols} is not a multiple of 16")
    if not eps >= 0.0:
        raise ValueError(f"eps must not be negative, got {eps}")
    device = x.device
    _require_cuda_device(device)
    h = x
    res_ptr = h_ptr = None
    if residual is not None:
        h = torch.empty_like(residual) if out_h is None else out_h
        res_ptr, h_ptr = residual.data_ptr(), h.data_ptr()
    rstd = _empty(rows, dtype=_F32, device=device) if save_rstd else None
    if fp8:
        codes = _empty((rows, cols), dtype=FP8_DTYPE, device=device)
        scale = _empty((rows, -(-cols // FP8_BLOCK)), dtype=_F32, device=device)
        y, y_ptr, y_elem, scale_ptr = FP8Tensor(codes, scale), codes.data_ptr(), 0, scale.data_ptr()
    else:
        y = _empty((rows, cols), dtype=out_dtype, device=device)
        y_ptr, y_elem, scale_ptr = y.data_ptr(), ELEM[out_dtype], None
    try:
        _call_on(device.index, "nf4_rmsnorm_fwd", x.data_ptr(), ELEM[x.dtype], res_ptr, ELEM[h.dtype],
                 weight.data_ptr(), ELEM[weight.dtype], rows, cols, eps, h_ptr, y_ptr, y_elem, scale_ptr,
                 None if rstd is None else rstd.data_ptr())
    except NF4Error as error:
        _refused(error, x=x, weight=weight, residual=residual, out_h=out_h)
    if out_h is not None:
        _written(out_h)
    return y, h, rstd


def nf4_rmsnorm_bwd(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                    dh: torch.Tensor | None = None):
    """The gradients of nf4_rmsnorm_fwd: (dx, dweight), dx [rows, cols] of h's
    type, the gradient of x and of the residual alike, dweight of weight's. dy
    is the gradient of y and dh (optional) the one that reaches h from the
    residual stream, both of h's type; h and rstd as the forward returned
    them. An 8-bit y passes its gradient through. Every tensor is contiguous
    and (rstd apart) starts on a 16-byte boundary."""
    if not _plain_matrix(h, weight):
        _check_norm(h, "h", weight)
    rows, cols = h.shape
    if not _like(dy, h):
        _require(dy, "dy", h.dtype, shape=h.shape)
        _same_device(h.device, dy=dy)
    if dh is not None and not _like(dh, h):
        _require(dh, "dh", h.dtype, shape=h.shape)
        _same_device(h.device, dh=dh)
    _require(rstd, "rstd", torch.float32, shape=(rows,))
    if rstd.device != h.device:
        _same_device(h.device, rstd=rstd)
    device = h.device
    _require_cuda_device(device)
    dx, dweight = torch.empty_like(h), torch.empty_like(weight)
    size = lib().nf4_rmsnorm_bwd_workspace(rows, cols)
    work = _empty(size, dtype=torch.uint8, device=device)
    try:
        _call_on(device.index, "nf4_rmsnorm_bwd", dy.data_ptr(), h.data_ptr(),
                 None if dh is None else dh.data_ptr(), ELEM[h.dtype], weight.data_ptr(),
                 ELEM[weight.dtype], rstd.data_ptr(), rows, cols, dx.data_ptr(), dweight.data_ptr(),
                 work.data_ptr(), size)
    except NF4Error as error:
        _refused(error, dy=dy, h=h, weight=weight, dh=dh)
    return dx, dweight
