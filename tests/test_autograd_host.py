"""The autograd wrappers' own logic on CPU tensors, with the library's calls
replaced by their formulas in torch: reshapes, casts, which gradient goes where,
second order."""
import types

import pytest
import torch

import dequant_gemm_gb300 as nf4
from dequant_gemm_gb300 import autograd as ag

EPS = 1e-6


@torch.no_grad()          # as the library, which autograd does not see into
def norm_fwd(x, weight, residual=None, eps=EPS, out_dtype=None, save_rstd=False, out_h=None):
    h = x if residual is None else (x.float() + residual.float()).to(residual.dtype)
    hd = h.double()
    rstd = torch.rsqrt(hd.square().mean(1) + eps)
    y = hd * rstd[:, None] * weight.double()
    return y.to(x.dtype if out_dtype in (None, torch.float8_e4m3fn) else out_dtype), h, rstd


@torch.no_grad()
def norm_bwd(dy, h, weight, rstd, dh=None):
    g, xh, r = dy.double() * weight.double(), h.double() * rstd[:, None], rstd[:, None]
    dx = r * (g - xh * (g * xh).mean(1, keepdim=True)) + (0 if dh is None else dh.double())
    return dx.to(h.dtype), (dy.double() * xh).sum(0).to(weight.dtype)


@pytest.fixture
def formulas(monkeypatch):
    """The library's calls as formulas; a weight is a namespace with its dense values."""
    @torch.no_grad()
    def fwd(x, w, out=None, out_dtype=torch.float32, accumulate=False):
        return (x.double() @ w.dense.double().t()).to(out_dtype)

    @torch.no_grad()
    def bwd(dy, w, out=None, out_dtype=torch.float32, accumulate=False):
        dx = (dy.double() @ w.dense.double()).to(out_dtype)
        return out.add_(dx) if accumulate else dx

    for name in ("nf4_matmul_fwd", "nf4_fp8_matmul_fwd"):
        monkeypatch.setattr(ag, name, fwd)
    for name in ("nf4_matmul_bwd_dx", "nf4_fp8_matmul_bwd_dx"):
        monkeypatch.setattr(ag, name, bwd)
    monkeypatch.setattr(ag, "nf4_fp8_quantize", lambda x, block_rows=1: x)
    monkeypatch.setattr(ag, "nf4_rmsnorm_fwd", norm_fwd)
    monkeypatch.setattr(ag, "nf4_rmsnorm_bwd", norm_bwd)


def rand(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def dense(rows, cols, seed):
    return types.SimpleNamespace(rows=rows, cols=cols, dense=rand(rows, cols, seed=seed))


@pytest.mark.parametrize("joined", [False, True])
@pytest.mark.parametrize("with_residual", [False, True])
def test_second_order_of_the_norm_is_refused(formulas, joined, with_residual):
    """The norm's gradients have no gradient of their own: a loss on them raises,
    also where another term gives it a graph and where the incoming gradient
    is a constant; first-order use with a graph asked for is the plain result."""
    x, w = rand(5, 32, seed=1).requires_grad_(), rand(32, seed=2).requires_grad_()
    res = rand(5, 32, seed=3).requires_grad_() if with_residual else None

    def loss():
        if joined:
            h, (y,) = ag.norm_fp8_linears(x, w, [dense(16, 32, 4)], residual=res, out_dtype=torch.float32)
        else:
            y, h = ag.rms_norm(x, w, res)
        return (y * rand(*y.shape, seed=5)).sum() + x.pow(3).sum()

    of = [x, w] + [res] * with_residual
    first = torch.autograd.grad(loss(), of)
    graph = torch.autograd.grad(loss(), of, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(first, graph))
    for g in graph:
        for t in of:
            with pytest.raises(RuntimeError, match="once"):
                torch.autograd.grad(g.square().sum(), t, retain_graph=True)


@pytest.mark.parametrize("kind", ["fp8", "nf4"])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_second_order_of_the_linear_layers(formulas, kind, out_dtype):
    """y = x W^T; for loss = sum(y^2) / 2 the gradient of <dL/dx, v> is W^T (W v),
    each product rounded as the wrappers round it. It does not depend on x."""
    w = dense(24, 32, 4)
    call = ag.fp8_linear if kind == "fp8" else ag.nf4_linear
    x, v = (rand(2, 3, 32, seed=s, dtype=torch.bfloat16) for s in (1, 2))
    x.requires_grad_()
    y = call(x, w, out_dtype)
    gx, = torch.autograd.grad(y.float().square().sum() / 2, x, create_graph=True)
    plain, = torch.autograd.grad(call(x, w, out_dtype).float().square().sum() / 2, x)
    assert torch.equal(gx, plain) and gx.dtype == x.dtype
    got, = torch.autograd.grad(gx, x, v, create_graph=True)
    once = (v.double() @ w.dense.double().t()).to(out_dtype)
    twice = once if kind == "fp8" else once.to(torch.bfloat16)
    assert torch.equal(got, (twice.double() @ w.dense.double()).bfloat16())
    third, = torch.autograd.grad(got.float().sum(), x, allow_unused=True)
    assert third is None or not third.any()


def test_second_order_of_nf4_linear_in_fp16(formulas):
    """An fp16 input: the gradient's own gradient has the output's type again."""
    w = dense(16, 64, 1)
    x, v = (rand(3, 64, seed=s, dtype=torch.float16) for s in (2, 3))
    x.requires_grad_()
    gx, = torch.autograd.grad(ag.nf4_linear(x, w).square().sum() / 2, x, create_graph=True)
    got, = torch.autograd.grad(gx, x, v)
    once = (v.double() @ w.dense.double().t()).float().half()
    assert torch.equal(got, (once.double() @ w.dense.double()).float().half())


def test_fp8_layer_keeps_its_buffers_types(monkeypatch):
    """A model converted to another type, moved or saved: codes and scales are
    neither parameters nor values of that type, and keep every bit."""
    def quantize(x, block_rows=1, out=None):
        assert block_rows == 128
        q = nf4.alloc_fp8(*x.shape, x.device, 128)
        q.codes.copy_(x), q.scale.copy_(rand(*q.scale.shape, seed=9))
        return q

    monkeypatch.setattr(ag, "nf4_fp8_quantize", quantize)
    layer = ag.FP8Linear(rand(160, 256, seed=1))
    codes, scale = layer.codes.view(torch.uint8).clone(), layer.scale.clone()
    model = torch.nn.Sequential(layer, torch.nn.Linear(160, 8))

    def same():
        w = layer.quantized_weight()
        return (w.codes.dtype == torch.float8_e4m3fn and torch.equal(w.codes.view(torch.uint8), codes)
                and torch.equal(w.scale, scale) and w.block_rows == 128)

    for convert in (lambda m: m.bfloat16(), lambda m: m.half(), lambda m: m.float(), lambda m: m.double(),
                    lambda m: m.to(torch.bfloat16), lambda m: m.to("cpu", torch.float16),
                    lambda m: m.type(torch.float32), lambda m: m.share_memory()):
        convert(model)
        assert same()
    assert model[1].weight.dtype == torch.float32
    state = {k: v.clone() for k, v in layer.state_dict().items()}
    assert {k: v.dtype for k, v in state.items()} == {"codes": torch.float8_e4m3fn, "scale": torch.float32}
    layer.codes.view(torch.uint8).zero_(), layer.scale.zero_()
    layer.load_state_dict(state)
    assert same()
    meta = layer.to("meta")
    assert meta.codes.device.type == "meta" and meta.codes.dtype == torch.float8_e4m3fn
    assert meta.scale.dtype == torch.float32


@pytest.mark.parametrize("dtype", ["nf4", "fp4", "int8"])
def test_nf4_layer_keeps_its_buffers_types(monkeypatch, dtype):
    """The same of the layer over 4-bit and int8 weights."""
    def quantize(W, out=None, dtype="nf4"):
        q = nf4.alloc_weight(*W.shape, W.device, dtype)
        q.codes.copy_(torch.arange(q.codes.numel()) % 100), q.absmax_scale.copy_(rand(*q.absmax_scale.shape, seed=9))
        if q.absmax_q is not None:
            q.absmax_q.copy_(torch.arange(q.absmax_q.numel()) % 200)
        return q

    monkeypatch.setattr(ag, "nf4_quantize", quantize)
    layer = ag.NF4Linear(rand(48, 128, seed=1), dtype=dtype)
    before = {k: v.clone() for k, v in layer.state_dict().items()}
    for convert in (lambda m: m.bfloat16(), lambda m: m.double(), lambda m: m.type(torch.float16), lambda m: m.to("cpu")):
        convert(torch.nn.Sequential(layer))
        now = layer.state_dict()
        assert now.keys() == before.keys()
        assert all(v.dtype == before[k].dtype and torch.equal(v, before[k]) for k, v in now.items())
        assert layer.quantized_weight().absmax_scale is layer.absmax_scale


def unaligned(*shape, seed=0, dtype=torch.float32):
    """A contiguous tensor that starts off a 16-byte boundary, as a row slice may."""
    n = 1
    for s in shape:
        n *= s
    t = rand(n + 1, seed=seed, dtype=dtype)[1:].view(shape)
    assert t.is_contiguous() and t.data_ptr() % 16
    return t


@pytest.mark.parametrize("cols, dtype", [(100, torch.bfloat16), (41, torch.float32)])
def test_norm_takes_tensors_off_the_16_byte_grid(formulas, monkeypatch, cols, dtype):
    """Row slices of odd widths, and gradients that come as slices of a larger
    one, reach the kernels on 16-byte boundaries, whatever their offset."""
    def strict(fn):
        def call(*args, **kw):
            for t in (*args, *kw.values()):
                assert not isinstance(t, torch.Tensor) or t.data_ptr() % 16 == 0 and t.is_contiguous()
            return fn(*args, **kw)
        return call

    for name in ("nf4_rmsnorm_fwd", "nf4_rmsnorm_bwd", "nf4_fp8_quantize", "nf4_matmul_fwd", "nf4_matmul_bwd_dx"):
        monkeypatch.setattr(ag, name, strict(getattr(ag, name)))
    x, res = unaligned(6, cols, seed=1, dtype=dtype), unaligned(6, cols, seed=2)
    w = unaligned(cols, seed=3)
    gy, gh = unaligned(6, cols, seed=4, dtype=dtype), unaligned(6, cols, seed=5)
    got, want = [], []
    for out, tensors in ((got, (x, w, res, gy, gh)), (want, [t.clone() for t in (x, w, res, gy, gh)])):
        x_, w_, r_ = (t.detach().requires_grad_() for t in tensors[:3])
        y, h = ag.rms_norm(x_, w_, r_)
        y2, _ = ag.rms_norm(x_, w_)
        out += [y, h, y2, *torch.autograd.grad([y, h, y2], [x_, w_, r_], [tensors[3], tensors[4], tensors[3]])]
        h, ys = ag.norm_fp8_linears(x_, w_, [dense(33, cols, 6), dense(9, cols, 7)], residual=r_, out_dtype=torch.float32)
        g = unaligned(6, 33, seed=8)
        out += [h, *ys, *torch.autograd.grad([h, ys[0], ys[1]], [x_, w_, r_], [tensors[4], g, g[:, :9]])]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_linear_layers_take_tensors_off_the_16_byte_grid(formulas, monkeypatch):
    def strict(t):
        assert t.data_ptr() % 16 == 0 and t.is_contiguous()
        return t

    quantize, fwd, bwd = ag.nf4_fp8_quantize, ag.nf4_matmul_fwd, ag.nf4_matmul_bwd_dx
    monkeypatch.setattr(ag, "nf4_fp8_quantize", lambda x, **kw: quantize(strict(x), **kw))
    monkeypatch.setattr(ag, "nf4_matmul_fwd", lambda x, w, **kw: fwd(strict(x), w, **kw))
    monkeypatch.setattr(ag, "nf4_matmul_bwd_dx", lambda x, w, **kw: bwd(strict(x), w, **kw))
    w = dense(50, 64, 4)
    for call in (ag.fp8_linear, ag.nf4_linear):
        x = unaligned(5, 64, seed=1, dtype=torch.bfloat16).requires_grad_()
        g = unaligned(5, 50, seed=2, dtype=torch.bfloat16)
        y = call(x, w, torch.bfloat16)
        gx, = torch.autograd.grad(y, x, g)
        x2 = x.detach().clone().requires_grad_()
        y2 = call(x2, w, torch.bfloat16)
        assert torch.equal(y, y2) and torch.equal(gx, torch.autograd.grad(y2, x2, g.clone())[0])


@pytest.mark.parametrize("joined", [False, True])
def test_residual_in_another_shape(formulas, joined):
    """A stream held as [tokens, width] beside x [batch, length, width]: its
    gradient has its own shape."""
    x, s, w = rand(2, 3, 32, seed=1, dtype=torch.bfloat16), rand(6, 32, seed=2), rand(32, seed=3)
    got = []
    for stream in (s, s.view(2, 3, 32)):
        x_, s_, w_ = (t.detach().clone().requires_grad_() for t in (x, stream, w))
        if joined:
            h, (y,) = ag.norm_fp8_linears(x_, w_, [dense(16, 32, 4)], residual=s_, out_dtype=torch.float32)
        else:
            y, h = ag.rms_norm(x_, w_, s_)
        assert h.shape == x.shape
        (h.square().sum() + y.float().sum()).backward()
        got.append([x_.grad, s_.grad.view(6, 32), w_.grad])
        assert s_.grad.shape == stream.shape
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("with_residual", [False, True])
def test_checkpointed_gradients(formulas, with_residual):
    """Recomputed in the backward pass (torch.utils.checkpoint) and with saved
    tensors packed away: the same gradients."""
    from torch.utils.checkpoint import checkpoint

    x, w, s = rand(2, 3, 32, seed=1), rand(32, seed=2), rand(2, 3, 32, seed=3)
    weights = [dense(16, 32, 4), dense(32, 32, 5)]

    def block(x, w, s):
        h, (a, b) = ag.norm_fp8_linears(x, w, weights, residual=s, out_dtype=torch.float32)
        y, h = ag.rms_norm(b, w, h if with_residual else None)
        return a.sum() + y.square().sum() + (0 if h is None else h.square().sum())

    def grads(run):
        t = [v.clone().requires_grad_() for v in (x, w, s)]
        args = (t[0], t[1], t[2] if with_residual else None)
        return torch.autograd.grad(run(*args), [v for v in args if v is not None])

    want = grads(block)
    with torch.autograd.graph.save_on_cpu():
        packed = grads(block)
    again = grads(lambda *a: checkpoint(block, *a, use_reentrant=False))
    for got in (packed, again):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
