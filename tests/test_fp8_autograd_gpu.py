"""The autograd wrappers of the 8-bit products and the RMS norm: they add only
reshapes and casts around the kernels, their gradients are the formulas' on the
rounded values, and the example block trains and decodes."""
import os
import sys

import pytest
import torch

import dequant_gemm_gb300 as nf4
from dequant_gemm_gb300.autograd import FP8Linear, fp8_linear, norm_fp8_linears, rms_norm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def rand(*shape, seed=0, std=1.0, dtype=torch.float32):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)


@pytest.mark.parametrize("lead", [(1,), (3, 7), (2, 90)])
def test_fp8_linear(lead):
    W = rand(384, 528, seed=1, std=0.02)
    layer = FP8Linear(W)
    assert list(layer.parameters()) == [] and set(layer.state_dict()) == {"codes", "scale"}
    w = layer.quantized_weight()
    x = rand(*lead, 528, seed=2, dtype=torch.bfloat16).requires_grad_(True)
    g = rand(*lead, 384, seed=3, std=0.1, dtype=torch.bfloat16)
    y = layer(x)
    y.backward(g)
    q = nf4.nf4_fp8_quantize(x.detach().reshape(-1, 528))
    assert torch.equal(y.reshape(-1, 384), nf4.nf4_fp8_matmul_fwd(q, w, out_dtype=torch.bfloat16))
    dq = nf4.nf4_fp8_quantize(g.reshape(-1, 384))
    assert torch.equal(x.grad.reshape(-1, 528), nf4.nf4_fp8_matmul_bwd_dx(dq, w, out_dtype=torch.bfloat16))
    assert fp8_linear(x.detach(), w).requires_grad is False


@pytest.mark.parametrize("dtype, res", [(torch.float32, torch.float32), (torch.bfloat16, torch.float32),
                                        (torch.bfloat16, None)])
def test_rms_norm_gradients(dtype, res):
    """Against torch's own autograd in fp64 on the same values: fp32 sums of
    100 terms, then the gradient's rounding to its type (2^-8 for bf16)."""
    x = rand(4, 9, 100, seed=1, dtype=dtype).requires_grad_(True)
    r = None if res is None else rand(4, 9, 100, seed=2, dtype=res).requires_grad_(True)
    w = (1 + rand(100, seed=3, std=0.1)).requires_grad_(True)
    gy, gh = rand(4, 9, 100, seed=4, dtype=dtype), rand(4, 9, 100, seed=5)
    y, h = rms_norm(x, w, r, 1e-5)
    loss = (y.float() * gy.float()).sum() + (0 if h is None else (h.float() * gh).sum())
    loss.backward()
    X, Wt = x.detach().double().requires_grad_(True), w.detach().double().requires_grad_(True)
    R = None if r is None else r.detach().double()
    H = X if R is None else X + R
    Y = H * torch.rsqrt((H * H).mean(-1, keepdim=True) + 1e-5) * Wt
    L = (Y * gy.double()).sum() + (0 if R is None else (H * gh.double()).sum())
    L.backward()
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    # a residual of 32 bits keeps h exact to 2^-24; the incoming gradients meet h's type
    scale = float(X.grad.abs().max())
    assert ((x.grad.double() - X.grad).abs() <= 2 * u * X.grad.abs() + 200 * 2.0 ** -24 * scale).all()
    assert ((w.grad.double() - Wt.grad).abs() <= 200 * 2.0 ** -24 * 36 * float(Wt.grad.abs().max())).all()
    if r is not None:
        assert r.grad.dtype == res


def test_norm_and_products_joined():
    x = rand(70, 528, seed=1, dtype=torch.bfloat16).requires_grad_(True)
    s = rand(70, 528, seed=2).requires_grad_(True)
    nw = (1 + rand(528, seed=3, std=0.1)).requires_grad_(True)
    ws = [nf4.nf4_fp8_quantize(rand(n, 528, seed=n, std=0.02), block_rows=128) for n in (256, 144)]
    h, ys = norm_fp8_linears(x, nw, ws, residual=s)
    gh, gys = rand(70, 528, seed=5), [rand(70, w.rows, seed=6, std=0.1, dtype=torch.bfloat16) for w in ws]
    torch.autograd.backward([h, *ys], [gh, *gys])
    q, h2, rstd = nf4.nf4_rmsnorm_fwd(x.detach(), nw.detach(), s.detach(), out_dtype=torch.float8_e4m3fn,
                                      save_rstd=True)
    assert torch.equal(h, h2)
    dy = None
    for y, g, w in zip(ys, gys, ws):
        assert torch.equal(y, nf4.nf4_fp8_matmul_fwd(q, w, out_dtype=torch.bfloat16))
        dy = nf4.nf4_fp8_matmul_bwd_dx(nf4.nf4_fp8_quantize(g), w, out=dy, accumulate=dy is not None)
    dx, dw = nf4.nf4_rmsnorm_bwd(dy, h2, nw.detach(), rstd, dh=gh)
    assert torch.equal(s.grad, dx) and torch.equal(x.grad, dx.bfloat16()) and torch.equal(nw.grad, dw)


def test_gradients_of_unused_outputs():
    """Only h, or only one product, takes part in the loss."""
    x, nw = rand(8, 256, seed=1).requires_grad_(True), torch.ones(256, device=DEV, requires_grad=True)
    ws = [nf4.nf4_fp8_quantize(rand(128, 256, seed=n, std=0.02), block_rows=128) for n in (1, 2)]
    h, ys = norm_fp8_linears(x, nw, ws)
    (h * 2).sum().backward()
    assert torch.equal(x.grad, torch.full_like(x, 2.0)) and not nw.grad.any()
    x.grad = None
    h, ys = norm_fp8_linears(x, nw, ws, out_dtype=torch.float32)
    ys[1].sum().backward()
    assert x.grad.abs().sum() > 0


def test_example_block():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        from fp8_mlp_block import run
    finally:
        sys.path.pop(0)
    off, losses, token, status = run(hidden=528, inner=1040, tokens=65, quiet=True)
    # three roundings to 3 mantissa bits on the way (two operands of each
    # product): well within a tenth of the output
    assert off < 0.1 and status == 0 and token.shape == (1, 528)
    assert all(b < a for a, b in zip(losses, losses[1:]))


@pytest.mark.parametrize("dx", [False, True], ids=["fwd", "dx"])
@pytest.mark.parametrize("M", [8, 100, 700])
def test_short_mma_wait_takes_the_abort_path_and_recovers(M, dx):
    """As for the 16-bit kernels: a short limit on a wait that completes anyway."""
    N, K = 2048, 1024
    w = nf4.nf4_fp8_quantize(rand(N, K, seed=1, std=0.02), block_rows=128)
    a = nf4.nf4_fp8_quantize(rand(M, N if dx else K, seed=2))
    fn = nf4.nf4_fp8_matmul_bwd_dx if dx else nf4.nf4_fp8_matmul_fwd
    want = fn(a, w)
    assert nf4.nf4_poll_device_status_site() == (0, 0)
    nf4.nf4_set_mma_wait_limit(200)
    try:
        fn(a, w)
        status, site = nf4.nf4_poll_device_status_site()
    finally:
        nf4.nf4_set_mma_wait_limit(0)
    assert status == 7 and (site & 0xffffffff) >> 28 == (5 if dx else 4) and (site >> 24) & 15 == 2
    assert torch.equal(fn(a, w), want) and nf4.nf4_poll_device_status_site() == (0, 0)


@pytest.mark.parametrize("joined", [False, True])
def test_second_order_of_the_norm_is_refused(joined):
    """Gradients asked for with a graph are the plain ones; a loss on them raises."""
    x, nw = rand(6, 256, seed=1).requires_grad_(True), (1 + rand(256, seed=2, std=0.1)).requires_grad_(True)
    w = nf4.nf4_fp8_quantize(rand(128, 256, seed=3, std=0.02), block_rows=128)

    def loss():
        y = norm_fp8_linears(x, nw, [w], out_dtype=torch.float32)[1][0] if joined else rms_norm(x, nw)[0]
        return (y * rand(*y.shape, seed=4)).sum() + x.pow(3).sum()

    plain = torch.autograd.grad(loss(), [x, nw])
    graph = torch.autograd.grad(loss(), [x, nw], create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(plain, graph))
    for g in graph:
        with pytest.raises(RuntimeError, match="once"):
            torch.autograd.grad(g.square().sum(), [x, nw], allow_unused=True)


def test_second_order_of_fp8_linear():
    """The gradient of <dL/dx, v> for L = sum(y^2) / 2 is dX(Y(v)), from the same calls."""
    w = nf4.nf4_fp8_quantize(rand(384, 528, seed=1, std=0.02), block_rows=128)
    x, v = rand(6, 528, seed=2, dtype=torch.bfloat16).requires_grad_(True), rand(6, 528, seed=3, dtype=torch.bfloat16)
    gx, = torch.autograd.grad(fp8_linear(x, w).float().square().sum() / 2, x, create_graph=True)
    got, = torch.autograd.grad(gx, x, v)
    u = nf4.nf4_fp8_matmul_fwd(nf4.nf4_fp8_quantize(v), w, out_dtype=torch.bfloat16)
    assert torch.equal(got, nf4.nf4_fp8_matmul_bwd_dx(nf4.nf4_fp8_quantize(u), w, out_dtype=torch.bfloat16))


def test_fp8_layer_in_a_converted_model():
    """A model taken to bf16, moved away and back: the layer gives the same bits."""
    layer = FP8Linear(rand(384, 528, seed=1, std=0.02))
    x = rand(5, 528, seed=2, dtype=torch.bfloat16)
    want = layer(x)
    model = torch.nn.Sequential(layer, torch.nn.Linear(384, 16, device=DEV))
    for convert in (lambda m: m.bfloat16(), lambda m: m.half(), lambda m: m.cpu().to(DEV), lambda m: m.float()):
        convert(model)
        assert torch.equal(layer(x), want)
    assert torch.equal(model.bfloat16()(x), model[1](want))


@pytest.mark.parametrize("cols, dtype", [(100, torch.bfloat16), (5001, torch.float32)])
def test_norm_of_row_slices_of_odd_widths(cols, dtype):
    """x[1:] starts off a 16-byte boundary, and so do gradients that come back as
    slices: the same bits as of copies, forward and backward."""
    x, s, w = rand(9, cols, seed=1, dtype=dtype), rand(9, cols, seed=2), 1 + rand(cols + 1, seed=3, std=0.1)
    gy, gh = rand(9, cols, seed=4, dtype=dtype), rand(9, cols, seed=5)
    got = []
    for part in (lambda t: t[1:], lambda t: t[1:].clone()):
        x_, s_, w_ = (part(t).detach().requires_grad_() for t in (x, s, w))
        y, h = rms_norm(x_, w_, s_)
        got.append([y, h, *torch.autograd.grad([y, h], [x_, s_, w_], [part(gy), part(gh)])])
    assert x[1:].data_ptr() % 16 and all(torch.equal(a, b) for a, b in zip(*got))


def test_gradients_as_slices_of_a_concatenation():
    """torch.cat hands its parts' gradients back as slices, here 200 bytes in."""
    x, w = rand(1, 100, seed=1).requires_grad_(True), torch.ones(100, device=DEV)
    parts = [rms_norm((x * k), w)[0].bfloat16() for k in (1.0, 2.0, 3.0)]
    torch.cat(parts).float().square().sum().backward()
    assert x.grad.isfinite().all()
    lead = rand(3, 528, seed=2, dtype=torch.bfloat16).requires_grad_(True)
    fw = nf4.nf4_fp8_quantize(rand(144, 528, seed=3, std=0.02), block_rows=128)
    torch.cat([fp8_linear(lead[:1], fw).float(), fp8_linear(lead[1:], fw).float()]).sum().backward()
    assert lead.grad.isfinite().all()
