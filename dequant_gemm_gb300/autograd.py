"""Frozen-base NF4 linear layer for PyTorch autograd.

The forward is the fused NF4-dequant matmul; the backward returns dL/dX through
the fused input-gradient kernel and no gradient for the quantized weight, which
is frozen ("Zenbit", zenbit.pallas_nf4 bullet: the backward computes dL/dX
only, without materialising the dequantized weight; "bitsandbytes", the layer
paragraph: a 4-bit linear layer over a quantized weight).

This module only marshals arguments: it flattens leading dimensions, casts the
incoming gradient to the input's type (bf16 or fp16, the kernels' activation
types) and the returned gradient to the input's dtype. Every product runs in
the library's kernels. Weights may be NF4, FP4 or int8 ("bitsandbytes", the
4-bit paragraph: Linear4bit / LinearNF4 / LinearFP4 layers; "Zenbit",
zenbit.int8 bullet).

The second half of the module does the same for the 8-bit floating point
products, the RMS norm in front of them and the gated block between them.
Rounding to 8 bits passes its gradient through; gradients of a product's output
are rounded to 8 bits themselves (1 x 128 blocks) before they meet the weight.

A backward pass can be captured into a CUDA graph. PyTorch ties a leaf's
accumulation to the stream of the graph that used it first: capture on leaves of
which no eager graph still lives (drop its outputs, or detach the leaves).
"""
from __future__ import annotations

import functools

import torch

from . import (FP8Tensor, NF4Weight, nf4_fp8_gated_bwd, nf4_fp8_gated_bwd_dx, nf4_fp8_gated_fwd,
               nf4_fp8_matmul_bwd_dx, nf4_fp8_matmul_fwd, nf4_fp8_quantize, nf4_matmul_bwd_dx,
               nf4_matmul_fwd, nf4_quantize, nf4_rmsnorm_bwd, nf4_rmsnorm_fwd)


def _aligned(t: torch.Tensor) -> torch.Tensor:
    """t contiguous and on a 16-byte boundary, as the kernels take it: a row slice
    of an odd width, as autograd itself passes them, need not start on one."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _matrix(t: torch.Tensor, cols: int) -> torch.Tensor:
    """t's rows of `cols` values as a matrix for the kernels."""
    return _aligned(t.reshape(-1, cols))


def _nf4_input_grad(gy, weight: NF4Weight, x_dtype, lead):
    gy2 = _aligned(gy.reshape(-1, weight.rows).to(x_dtype))
    # a bf16 input gets its gradient straight from the kernel's bf16 output
    out = torch.bfloat16 if x_dtype == torch.bfloat16 else torch.float32
    gx = nf4_matmul_bwd_dx(gy2, weight, out_dtype=out)
    return gx.reshape(*lead, weight.cols).to(x_dtype)


class NF4InputGradFunction(torch.autograd.Function):
    """NF4LinearFunction's gradient as a function of the incoming one, to which
    it is linear; its own gradient is the product again."""

    @staticmethod
    def forward(ctx, gy, weight: NF4Weight, x_dtype, lead):
        ctx.weight, ctx.gy_dtype = weight, gy.dtype
        return _nf4_input_grad(gy, weight, x_dtype, lead)

    @staticmethod
    def backward(ctx, v):
        return NF4LinearFunction.apply(v, ctx.weight, ctx.gy_dtype), None, None, None


class NF4LinearFunction(torch.autograd.Function):
    """y = x · dequant(W)ᵀ for bf16 or fp16 x [..., cols] -> y [..., rows] of
    `out_dtype` (fp32 or bf16); differentiable in x, any number of times."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, weight: NF4Weight,
                out_dtype: torch.dtype = torch.float32) -> torch.Tensor:
        if x.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"x must be bfloat16 or float16, got {x.dtype}")
        if x.shape[-1] != weight.cols:
            raise ValueError(f"x must end in {weight.cols} features, got {tuple(x.shape)}")
        lead = x.shape[:-1]
        y = nf4_matmul_fwd(_matrix(x, weight.cols), weight, out_dtype=out_dtype)
        ctx.weight = weight
        ctx.lead = lead
        ctx.x_dtype = x.dtype
        return y.reshape(*lead, weight.rows)

    @staticmethod
    def backward(ctx, gy: torch.Tensor):
        if not ctx.needs_input_grad[0]:
            return None, None, None
        # under create_graph the result is a function of gy
        grad = NF4InputGradFunction.apply if torch.is_grad_enabled() else _nf4_input_grad
        return grad(gy, ctx.weight, ctx.x_dtype, ctx.lead), None, None


def nf4_linear(x: torch.Tensor, weight: NF4Weight,
               out_dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """Differentiable in x; the quantized weight gets no gradient."""
    return NF4LinearFunction.apply(x, weight, out_dtype)


class _Frozen(torch.nn.Module):
    """A layer whose buffers named in `_frozen` keep their types and bits when the
    module is converted to another type (.to(dtype), .half() and the like, which
    would round codes and scales): they only move."""
    _frozen = ()

    def _apply(self, fn, recurse=True):
        kept = {n: self._buffers[n] for n in self._frozen if self._buffers.get(n) is not None}
        as_bits = {n: t.view({1: torch.uint8, 4: torch.int32}[t.element_size()]) for n, t in kept.items()}
        self._buffers.update(as_bits)        # whole numbers: not converted with floating-point types
        try:
            super()._apply(fn, recurse)
            for n, t in as_bits.items():
                moved = self._buffers[n]     # .type(dtype) converts whole numbers too
                kept[n] = (moved if moved.dtype == t.dtype else t.to(moved.device)).view(kept[n].dtype)
        finally:
            self._buffers.update(kept)
        return self


class NF4Linear(_Frozen):
    """A frozen linear layer (no bias) holding its weight quantized (NF4 by
    default; "fp4" or "int8" on request).

    The codes and scales are buffers: they move with the module and are saved
    in its state dict, no optimizer sees them and no conversion of the module
    changes them."""
    _frozen = ("codes", "absmax_q", "absmax_scale")

    def __init__(self, weight: torch.Tensor, dtype: str = "nf4",
                 out_dtype: torch.dtype = torch.float32):
        super().__init__()
        if weight.dim() != 2:
            raise ValueError("weight must be 2-D [out_features, in_features]")
        w = weight.detach()
        if w.dtype not in (torch.float32, torch.bfloat16):
            w = w.to(torch.float32)
        q = nf4_quantize(_aligned(w), dtype=dtype)
        self.register_buffer("codes", q.codes)
        if q.absmax_q is not None:
            self.register_buffer("absmax_q", q.absmax_q)
        else:
            self.absmax_q = None
        self.register_buffer("absmax_scale", q.absmax_scale)
        self.out_features, self.in_features = q.rows, q.cols
        self.qdtype = dtype
        self.out_dtype = out_dtype

    def quantized_weight(self) -> NF4Weight:
        return NF4Weight(self.codes, self.absmax_q, self.absmax_scale, self.out_features,
                         self.in_features, self.qdtype)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return nf4_linear(x, self.quantized_weight(), self.out_dtype)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, "
                f"{self.qdtype}")


class _Once(torch.autograd.Function):
    """A gradient g that depends on `inputs`, in a way that has no gradient."""

    @staticmethod
    def forward(ctx, g, *inputs):
        return g.view_as(g)

    @staticmethod
    def backward(ctx, gg):
        raise RuntimeError("the gradients of the RMS norm and of the gated block can be taken once: they are "
                           "not differentiable themselves (second-order gradients)")


def _once(backward):
    """A Function's backward whose results no later backward pass may go through.
    Under create_graph they would be constants in autograd's eyes, and a loss on
    them would lack, without an error, all that comes of the saved tensors; so
    they get a graph to these (which have to be the Function's own inputs or
    outputs) and to the incoming gradients, one that raises. (torch's
    once_differentiable does so only where the incoming gradients need one, and
    not on the way to the Function's inputs.)"""
    @functools.wraps(backward)
    def run(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return out
        inputs = [t for t in (*ctx.saved_tensors, *grads) if t is not None and t.requires_grad]
        return tuple(None if g is None else _Once.apply(g, *inputs) for g in out)
    return run


class RMSNormFunction(torch.autograd.Function):
    """(y, h) with h = x + residual and y = h / rms(h) * weight, y of x's type.
    Without a residual h is not returned (None)."""

    @staticmethod
    def forward(ctx, x, weight, residual=None, eps=1e-6):
        shape = x.shape
        rows = _matrix(x, shape[-1])
        res = None if residual is None else _aligned(residual.reshape(rows.shape))
        y, h, rstd = nf4_rmsnorm_fwd(rows, _aligned(weight), res, eps=eps, save_rstd=True)
        h = x if residual is None else h.reshape(shape)
        ctx.save_for_backward(h, weight, rstd)       # h: this Function's own input or output (_once)
        ctx.x_dtype = x.dtype
        ctx.res_shape = None if residual is None else residual.shape
        return y.reshape(shape), (h if residual is not None else None)

    @staticmethod
    @_once
    def backward(ctx, gy, gh):
        h, weight, rstd = ctx.saved_tensors
        h = _matrix(h, h.shape[-1])
        flat = lambda g: None if g is None else _aligned(g.reshape(h.shape).to(h.dtype))  # noqa: E731
        dx, dweight = nf4_rmsnorm_bwd(flat(gy), h, _aligned(weight), rstd, dh=flat(gh))
        dx = dx.reshape(gy.shape)
        return dx.to(ctx.x_dtype), dweight, (dx.reshape(ctx.res_shape) if ctx.res_shape else None), None


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
             eps: float = 1e-6):
    """Differentiable RMS norm with the residual's addition: (y, h), h None
    without a residual."""
    return RMSNormFunction.apply(x, weight, residual, eps)


def _fp8_input_grad(gy, weight: FP8Tensor, x_dtype, shape):
    q = nf4_fp8_quantize(_matrix(gy, weight.rows))
    out = torch.bfloat16 if x_dtype == torch.bfloat16 else torch.float32
    return nf4_fp8_matmul_bwd_dx(q, weight, out_dtype=out).reshape(shape).to(x_dtype)


class FP8InputGradFunction(torch.autograd.Function):
    """FP8LinearFunction's gradient as a function of the incoming one, to which
    it is linear; its own gradient is the product again."""

    @staticmethod
    def forward(ctx, gy, weight: FP8Tensor, x_dtype, shape):
        ctx.weight, ctx.gy_dtype = weight, gy.dtype
        return _fp8_input_grad(gy, weight, x_dtype, shape)

    @staticmethod
    def backward(ctx, v):
        return FP8LinearFunction.apply(v, ctx.weight, ctx.gy_dtype), None, None, None


class FP8LinearFunction(torch.autograd.Function):
    """y = x · value(weight)ᵀ, x [..., cols] (fp32, bf16 or fp16) rounded to 8
    bits, y of `out_dtype` (fp32 or bf16); differentiable in x, any number of
    times."""

    @staticmethod
    def forward(ctx, x, weight: FP8Tensor, out_dtype=torch.bfloat16):
        ctx.weight, ctx.x_dtype, ctx.shape = weight, x.dtype, x.shape
        q = nf4_fp8_quantize(_matrix(x, x.shape[-1]))
        return nf4_fp8_matmul_fwd(q, weight, out_dtype=out_dtype).reshape(*x.shape[:-1], weight.rows)

    @staticmethod
    def backward(ctx, gy):
        if not ctx.needs_input_grad[0]:
            return None, None, None
        # under create_graph the result is a function of gy
        grad = FP8InputGradFunction.apply if torch.is_grad_enabled() else _fp8_input_grad
        return grad(gy, ctx.weight, ctx.x_dtype, ctx.shape), None, None


def fp8_linear(x: torch.Tensor, weight: FP8Tensor,
               out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    return FP8LinearFunction.apply(x, weight, out_dtype)


class NormFP8LinearsFunction(torch.autograd.Function):
    """The norm and the products that read its output, joined: the norm writes
    the 8-bit operand once for all weights. Returns (h, y_0, y_1, ...)."""

    @staticmethod
    def forward(ctx, x, norm_weight, residual, eps, out_dtype, *weights):
        shape = x.shape
        rows = _matrix(x, shape[-1])
        res = None if residual is None else _aligned(residual.reshape(rows.shape))
        q, h, rstd = nf4_rmsnorm_fwd(rows, _aligned(norm_weight), res, eps=eps,
                                     out_dtype=torch.float8_e4m3fn, save_rstd=True)
        h = x if residual is None else h.reshape(shape)
        ctx.save_for_backward(h, norm_weight, rstd)  # h: this Function's own input or output (_once)
        ctx.weights, ctx.x_dtype, ctx.shape = weights, x.dtype, shape
        ctx.res_shape = None if residual is None else residual.shape
        ctx.set_materialize_grads(False)     # an output that nothing used costs no product
        ys = [nf4_fp8_matmul_fwd(q, w, out_dtype=out_dtype).reshape(*shape[:-1], w.rows)
              for w in weights]
        # an output may not be the input itself
        return (h.clone() if residual is None else h, *ys)

    @staticmethod
    @_once
    def backward(ctx, gh, *gys):
        h, norm_weight, rstd = ctx.saved_tensors
        h = _matrix(h, h.shape[-1])
        dy = None                    # the products' input gradients, summed in fp32
        for w, g in zip(ctx.weights, gys):
            if g is not None:
                q = nf4_fp8_quantize(_matrix(g, w.rows))
                dy = nf4_fp8_matmul_bwd_dx(q, w, out=dy, accumulate=dy is not None)
        dy = torch.zeros_like(h) if dy is None else dy.to(h.dtype)
        dh = None if gh is None else _aligned(gh.reshape(h.shape).to(h.dtype))
        dx, dweight = nf4_rmsnorm_bwd(dy, h, _aligned(norm_weight), rstd, dh=dh)
        dx = dx.reshape(ctx.shape)
        return (dx.to(ctx.x_dtype), dweight, dx.reshape(ctx.res_shape) if ctx.res_shape else None, None, None,
                *[None] * len(ctx.weights))


def norm_fp8_linears(x: torch.Tensor, norm_weight: torch.Tensor, weights, residual=None,
                     eps: float = 1e-6, out_dtype: torch.dtype = torch.bfloat16):
    """h = x + residual and, for each 8-bit weight, rms_norm(h) · value(weight)ᵀ:
    (h, [y, ...]). Differentiable in x, the residual and the norm's weight."""
    h, *ys = NormFP8LinearsFunction.apply(x, norm_weight, residual, eps, out_dtype, *weights)
    return h, ys


class FP8Linear(_Frozen):
    """A frozen linear layer (no bias) holding its weight in 8 bits, with a
    scale for each 128 x 128 block. Codes and scales are buffers, which no
    conversion of the module changes."""
    _frozen = ("codes", "scale")

    def __init__(self, weight: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16):
        super().__init__()
        if weight.dim() != 2:
            raise ValueError("weight must be 2-D [out_features, in_features]")
        q = nf4_fp8_quantize(_aligned(weight.detach()), block_rows=128)
        self.register_buffer("codes", q.codes)
        self.register_buffer("scale", q.scale)
        self.out_features, self.in_features = q.rows, q.cols
        self.out_dtype = out_dtype

    def quantized_weight(self) -> FP8Tensor:
        return FP8Tensor(self.codes, self.scale, 128)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return fp8_linear(x, self.quantized_weight(), self.out_dtype)

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, out_features={self.out_features}, fp8"


# The block keeps its projections for the backward pass (4 bytes a value of theirs)
# where a graph is recorded. A Function cannot see that: in its forward the gradient
# mode is off, and needs_input_grad says what its inputs require in any mode. The
# wrappers hand it in as `graph`.


def _gated_mlp(q: FP8Tensor, gate, up, down, activation, out_dtype, keep: bool):
    """(y, g, u): y of an 8-bit operand, g and u what its gradient needs (None unless keep)."""
    a, g, u = nf4_fp8_gated_fwd(q, gate, up, activation=activation, save=keep)
    return nf4_fp8_matmul_fwd(a, down, out_dtype=out_dtype), g, u


def _gated_mlp_grad(gy, g, u, gate, up, down, activation, out_dtype):
    """The gradient of the 8-bit operand's values, [M, cols] of out_dtype (fp32 or bf16)."""
    da = nf4_fp8_matmul_bwd_dx(nf4_fp8_quantize(_matrix(gy, down.rows)), down, out_dtype=out_dtype)
    return nf4_fp8_gated_bwd_dx(*nf4_fp8_gated_bwd(da, g, u, activation=activation), gate, up, out_dtype=out_dtype)


class FP8GatedMLPFunction(torch.autograd.Function):
    """y = (act(x gate^T) * (x up^T)) down^T, x [..., cols] (fp32, bf16 or fp16)
    and the product in front of down rounded to 8 bits, y of `out_dtype` (fp32 or
    bf16); differentiable in x, once. Returns (y, g): the gradient does not read x,
    which is not kept (it may change in place); the projection g, an output for that
    reason alone, ties the graph that raises to x (_once)."""

    @staticmethod
    def forward(ctx, x, gate, up, down, activation="silu", out_dtype=torch.bfloat16, graph=True):
        ctx.weights, ctx.activation = (gate, up, down), activation
        keep = graph and ctx.needs_input_grad[0]
        q = nf4_fp8_quantize(_matrix(x, x.shape[-1]))
        y, g, u = _gated_mlp(q, gate, up, down, activation, out_dtype, keep)
        ctx.x_dtype, ctx.shape = x.dtype, x.shape
        ctx.set_materialize_grads(False)     # (g's is None)
        if keep:
            ctx.save_for_backward(g, u)
        return y.reshape(*x.shape[:-1], down.rows), g

    @staticmethod
    @_once
    def backward(ctx, gy, _):
        g, u = ctx.saved_tensors
        if gy is None:
            return torch.zeros(ctx.shape, dtype=ctx.x_dtype, device=g.device), *[None] * 6
        out = torch.bfloat16 if ctx.x_dtype == torch.bfloat16 else torch.float32
        dx = _gated_mlp_grad(gy, g, u, *ctx.weights, ctx.activation, out)
        return dx.reshape(ctx.shape).to(ctx.x_dtype), *[None] * 6


def fp8_gated_mlp(x: torch.Tensor, gate: FP8Tensor, up: FP8Tensor, down: FP8Tensor, activation: str = "silu",
                  out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The gated feed-forward block on frozen 8-bit weights; differentiable in x."""
    return FP8GatedMLPFunction.apply(x, gate, up, down, activation, out_dtype, torch.is_grad_enabled())[0]


class NormFP8GatedMLPFunction(torch.autograd.Function):
    """The norm and the gated block that reads its output, joined: (h, y)."""

    @staticmethod
    def forward(ctx, x, norm_weight, residual, eps, gate, up, down, activation, out_dtype, graph=True):
        shape = x.shape
        rows = _matrix(x, shape[-1])
        res = None if residual is None else _aligned(residual.reshape(rows.shape))
        q, h, rstd = nf4_rmsnorm_fwd(rows, _aligned(norm_weight), res, eps=eps,
                                     out_dtype=torch.float8_e4m3fn, save_rstd=True)
        h = x if residual is None else h.reshape(shape)
        keep = graph and any(ctx.needs_input_grad[:3])
        y, g, u = _gated_mlp(q, gate, up, down, activation, out_dtype, keep)
        ctx.weights, ctx.activation, ctx.x_dtype, ctx.shape = (gate, up, down), activation, x.dtype, shape
        ctx.res_shape = None if residual is None else residual.shape
        ctx.set_materialize_grads(False)     # an output that nothing used costs no product
        if keep:
            ctx.save_for_backward(h, norm_weight, rstd, g, u)    # h: this Function's own input or output (_once)
        # an output may not be the input itself
        return (h.clone() if residual is None else h), y.reshape(*shape[:-1], down.rows)

    @staticmethod
    @_once
    def backward(ctx, gh, gy):
        h, norm_weight, rstd, g, u = ctx.saved_tensors
        h = _matrix(h, h.shape[-1])
        if gy is None:
            dy = torch.zeros_like(h)
        else:
            out = torch.bfloat16 if h.dtype == torch.bfloat16 else torch.float32
            dy = _gated_mlp_grad(gy, g, u, *ctx.weights, ctx.activation, out).to(h.dtype)
        dh = None if gh is None else _aligned(gh.reshape(h.shape).to(h.dtype))
        dx, dweight = nf4_rmsnorm_bwd(dy, h, _aligned(norm_weight), rstd, dh=dh)
        dx = dx.reshape(ctx.shape)
        return (dx.to(ctx.x_dtype), dweight, dx.reshape(ctx.res_shape) if ctx.res_shape else None,
                *[None] * 7)


def norm_fp8_gated_mlp(x: torch.Tensor, norm_weight: torch.Tensor, gate: FP8Tensor, up: FP8Tensor,
                       down: FP8Tensor, residual=None, eps: float = 1e-6, activation: str = "silu",
                       out_dtype: torch.dtype = torch.bfloat16):
    """h = x + residual and the gated block of rms_norm(h): (h, y). Differentiable in
    x, the residual and the norm's weight."""
    return NormFP8GatedMLPFunction.apply(x, norm_weight, residual, eps, gate, up, down, activation, out_dtype,
                                         torch.is_grad_enabled())


class FP8GatedMLP(_Frozen):
    """A frozen gated feed-forward block (no biases) holding its three weights in
    8 bits: gate and up [inner, features], down [features_out, inner]."""
    _frozen = tuple(f"{n}_{part}" for n in ("gate", "up", "down") for part in ("codes", "scale"))

    def __init__(self, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor, activation: str = "silu",
                 out_dtype: torch.dtype = torch.bfloat16):
        super().__init__()
        if gate.dim() != 2 or gate.shape != up.shape or down.dim() != 2 or down.shape[1] != gate.shape[0]:
            raise ValueError("gate and up must be [inner, features] and down [features_out, inner], got "
                             f"{tuple(gate.shape)}, {tuple(up.shape)} and {tuple(down.shape)}")
        for name, w in (("gate", gate), ("up", up), ("down", down)):
            q = nf4_fp8_quantize(_aligned(w.detach()), block_rows=128)
            self.register_buffer(f"{name}_codes", q.codes)
            self.register_buffer(f"{name}_scale", q.scale)
        self.in_features, self.inner_features, self.out_features = gate.shape[1], gate.shape[0], down.shape[0]
        self.activation, self.out_dtype = activation, out_dtype

    def quantized_weights(self) -> tuple[FP8Tensor, FP8Tensor, FP8Tensor]:
        """(gate, up, down)"""
        return tuple(FP8Tensor(getattr(self, f"{n}_codes"), getattr(self, f"{n}_scale"), 128)
                     for n in ("gate", "up", "down"))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return fp8_gated_mlp(x, *self.quantized_weights(), self.activation, self.out_dtype)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, inner_features={self.inner_features}, "
                f"out_features={self.out_features}, {self.activation}, fp8")
