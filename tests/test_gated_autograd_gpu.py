"""The gated block's autograd wrappers add only reshapes and casts around the
kernels; its gradients are the formulas'; a training step of it with the other
operators, back to back and in CUDA graphs, and a decoding step on 4-bit weights."""
import pytest
import torch
import torch.utils.checkpoint

import dequant_gemm_gb300 as nf4
from dequant_gemm_gb300.autograd import FP8GatedMLP, fp8_gated_mlp, norm_fp8_gated_mlp

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8, F32, BF16, F16 = torch.float8_e4m3fn, torch.float32, torch.bfloat16, torch.float16


def rand(*shape, seed=0, std=1.0, dtype=F32):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)


def weights(inner=400, features=528, out=272):
    return rand(inner, features, seed=1, std=0.02), rand(inner, features, seed=2, std=0.02), rand(out, inner, seed=3, std=0.02)


@pytest.mark.parametrize("activation", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("lead", [(1,), (3, 7), (2, 90)])
def test_module(lead, dtype, activation):
    mlp = FP8GatedMLP(*weights(), activation=activation)
    assert list(mlp.parameters()) == [] and len(mlp.state_dict()) == 6
    gate, up, down = mlp.quantized_weights()
    x = rand(*lead, 528, seed=4, dtype=dtype).requires_grad_(True)
    y = mlp(x)
    gy = rand(*lead, 272, seed=5, std=0.1, dtype=BF16)
    y.backward(gy)
    q = nf4.nf4_fp8_quantize(x.detach().reshape(-1, 528))
    a, g, u = nf4.nf4_fp8_gated_fwd(q, gate, up, activation=activation, save=True)
    assert y.dtype == BF16 and torch.equal(y.reshape(-1, 272), nf4.nf4_fp8_matmul_fwd(a, down, out_dtype=BF16))
    t = BF16 if dtype == BF16 else F32
    da = nf4.nf4_fp8_matmul_bwd_dx(nf4.nf4_fp8_quantize(gy.reshape(-1, 272)), down, out_dtype=t)
    dx = nf4.nf4_fp8_gated_bwd_dx(*nf4.nf4_fp8_gated_bwd(da, g, u, activation=activation), gate, up, out_dtype=t)
    assert x.grad.dtype == dtype and torch.equal(x.grad.reshape(-1, 528), dx.to(dtype))
    assert mlp(x.detach()).requires_grad is False


def test_gradient_against_torch_autograd():
    """The block in 64 bits on the 8-bit weights' values. What the kernels round: x,
    a and the gradients dy, dG, dU to 8 bits (2^-4 of a value at most, 2^-10 of the
    block's largest / 448 below), G and U to bf16 (2^-8). Each enters the gradient
    linearly; with independent signs over 400 and 272 terms the relative error of
    the whole is below the sum of the largest single ones: 4 * 2^-4 + 3 * 2^-8."""
    mlp = FP8GatedMLP(*weights())
    x, gy = rand(60, 528, seed=4).requires_grad_(True), rand(60, 272, seed=5)
    mlp(x).backward(gy.bfloat16())
    gate, up, down = (nf4.nf4_fp8_dequantize(w).double() for w in mlp.quantized_weights())
    X = x.detach().double().requires_grad_(True)
    Y = (torch.nn.functional.silu(X @ gate.t()) * (X @ up.t())) @ down.t()
    Y.backward(gy.bfloat16().double())
    assert float((x.grad.double() - X.grad).norm() / X.grad.norm()) <= 4 * 2.0 ** -4 + 3 * 2.0 ** -8


@pytest.mark.parametrize("with_residual", [False, True])
def test_norm_and_block_joined(with_residual):
    gate, up, down = FP8GatedMLP(*weights()).quantized_weights()
    x = rand(70, 528, seed=1, dtype=BF16).requires_grad_(True)
    s = rand(70, 528, seed=2).requires_grad_(True) if with_residual else None
    nw = (1 + rand(528, seed=3, std=0.1)).requires_grad_(True)
    h, y = norm_fp8_gated_mlp(x, nw, gate, up, down, residual=s)
    gh, gy = rand(70, 528, seed=5, dtype=h.dtype), rand(70, 272, seed=6, std=0.1, dtype=BF16)
    torch.autograd.backward([h, y], [gh, gy])
    q, h2, rstd = nf4.nf4_rmsnorm_fwd(x.detach(), nw.detach(), None if s is None else s.detach(), out_dtype=F8,
                                      save_rstd=True)
    a, g, u = nf4.nf4_fp8_gated_fwd(q, gate, up, save=True)
    assert torch.equal(h, h2) and torch.equal(y, nf4.nf4_fp8_matmul_fwd(a, down, out_dtype=BF16))
    t = F32 if with_residual else BF16
    da = nf4.nf4_fp8_matmul_bwd_dx(nf4.nf4_fp8_quantize(gy), down, out_dtype=t)
    dn = nf4.nf4_fp8_gated_bwd_dx(*nf4.nf4_fp8_gated_bwd(da, g, u), gate, up, out_dtype=t)
    dx, dw = nf4.nf4_rmsnorm_bwd(dn, h2, nw.detach(), rstd, dh=gh)
    assert torch.equal(x.grad, dx.bfloat16()) and torch.equal(nw.grad, dw)
    assert s is None or torch.equal(s.grad, dx)


def test_gradients_of_unused_outputs():
    gate, up, down = FP8GatedMLP(*weights()).quantized_weights()
    x, nw = rand(8, 528, seed=1).requires_grad_(True), torch.ones(528, device=DEV, requires_grad=True)
    h, y = norm_fp8_gated_mlp(x, nw, gate, up, down)
    (h * 2).sum().backward()
    assert torch.equal(x.grad, torch.full_like(x, 2.0)) and not nw.grad.any()
    x.grad = None
    norm_fp8_gated_mlp(x, nw, gate, up, down, out_dtype=F32)[1].sum().backward()
    assert x.grad.abs().sum() > 0
    # nothing is kept where no gradient is wanted
    h, y = norm_fp8_gated_mlp(x.detach(), nw.detach(), gate, up, down)
    assert not y.requires_grad and not h.requires_grad


@pytest.mark.parametrize("joined", [False, True])
def test_second_order_is_refused(joined):
    gate, up, down = FP8GatedMLP(*weights()).quantized_weights()
    x, nw = rand(6, 528, seed=1).requires_grad_(True), (1 + rand(528, seed=2, std=0.1)).requires_grad_(True)

    def loss():
        y = norm_fp8_gated_mlp(x, nw, gate, up, down, out_dtype=F32)[1] if joined else \
            fp8_gated_mlp(x, gate, up, down, out_dtype=F32)
        return (y * rand(*y.shape, seed=4)).sum() + x.pow(3).sum()

    of = [x, nw] if joined else [x]
    plain = torch.autograd.grad(loss(), of)
    graph = torch.autograd.grad(loss(), of, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(plain, graph))
    for g in graph:
        with pytest.raises(RuntimeError, match="once"):
            torch.autograd.grad(g.square().sum(), of, allow_unused=True)


def test_converted_and_checkpointed():
    """A model taken to other types and away and back gives the same bits; so does a
    checkpointed one."""
    mlp = FP8GatedMLP(*weights())
    x = rand(5, 528, seed=2, dtype=BF16).requires_grad_(True)
    want, = torch.autograd.grad(mlp(x).float().square().sum(), x)
    model = torch.nn.Sequential(mlp, torch.nn.Linear(272, 16, device=DEV))
    for convert in (lambda m: m.bfloat16(), lambda m: m.half(), lambda m: m.cpu().to(DEV), lambda m: m.float()):
        convert(model)
        got, = torch.autograd.grad(mlp(x).float().square().sum(), x)
        assert torch.equal(got, want)
    y = torch.utils.checkpoint.checkpoint(mlp, x, use_reentrant=False)
    assert torch.equal(torch.autograd.grad(y.float().square().sum(), x)[0], want)


def test_tensors_off_the_16_byte_grid():
    mlp = FP8GatedMLP(*weights())
    big = rand(1 + 9 * 528, seed=1, dtype=F32)
    got = []
    for x in (big[1:].view(9, 528), big[1:].clone().view(9, 528)):
        x = x.detach().requires_grad_()
        got.append(torch.autograd.grad(mlp(x).float().square().sum(), x)[0])
    assert torch.equal(*got)


def training_step(s, wait):
    """A block's forward and backward with its neighbours, the weights quantized within it."""
    out = []

    def did(*ts):
        for t in ts:
            out.extend([t.codes.view(torch.uint8), t.scale] if isinstance(t, nf4.FP8Tensor) else [t])
        if wait:
            torch.cuda.synchronize()
        return ts[0] if len(ts) == 1 else ts

    gate, up, down = (did(nf4.nf4_fp8_quantize(s[n], block_rows=128)) for n in ("gate", "up", "down"))
    q, h, rstd = did(*nf4.nf4_rmsnorm_fwd(s["x"], s["norm"], s["stream"], out_dtype=F8, save_rstd=True))
    a, g, u = did(*nf4.nf4_fp8_gated_fwd(q, gate, up, activation="gelu_tanh", save=True))
    y = did(nf4.nf4_fp8_matmul_fwd(a, down, out_dtype=BF16))
    da = did(nf4.nf4_fp8_matmul_bwd_dx(did(nf4.nf4_fp8_quantize(y)), down, out_dtype=BF16))
    dg, du = did(*nf4.nf4_fp8_gated_bwd(da, g, u, activation="gelu_tanh"))
    dn = did(nf4.nf4_fp8_gated_bwd_dx(dg, du, gate, up))
    did(*nf4.nf4_rmsnorm_bwd(dn, h, s["norm"], rstd))
    return out


def decoding_step(s, wait):
    """The same block's decoding on 4-bit weights, quantized within it."""
    out = []

    def did(*ts):
        out.extend(t for t in ts if t is not None)
        if wait:
            torch.cuda.synchronize()

    ws = []
    for n in ("gate", "up", "down"):
        w = nf4.nf4_int4_quantize(s[n], group=32 if n == "down" else 64, zero_point=n != "up")
        did(w.codes, w.scale, w.zero)
        ws.append(w)
    n, h, _ = nf4.nf4_rmsnorm_fwd(s["x"], s["norm"], s["stream"])
    did(n, h)
    a = nf4.nf4_int4_gated_fwd(n, ws[0], ws[1])
    did(a)
    y = nf4.nf4_int4_matmul_fwd(a, ws[2], out_dtype=BF16)
    did(y)
    did(nf4.nf4_int4_dequantize(ws[2], out_dtype=BF16))
    nf4.nf4_int4_matmul_fwd(a, ws[2], out=(z := h.clone()), accumulate=True)
    did(z)
    return out


def inputs(M, seed):
    return {"x": rand(M, 576, seed=seed, dtype=BF16), "stream": rand(M, 576, seed=seed + 1),
            "norm": 1 + rand(576, seed=seed + 2, std=0.1), "gate": rand(1056, 576, seed=seed + 3, std=0.02),
            "up": rand(1056, 576, seed=seed + 4, std=0.02), "down": rand(576, 1056, seed=seed + 5, std=0.02)}


@pytest.mark.parametrize("M, step", [(1, training_step), (40, training_step), (300, training_step), (1, decoding_step),
                                     (6, decoding_step), (20, decoding_step)])
def test_steps_back_to_back_and_in_graphs(M, step):
    """Bits as with a synchronisation after every call; two graphs of the same step
    on two streams at once, each with tensors of its own."""
    batches = [inputs(M, 10 * k) for k in range(1, 5)]
    want = [step(s, True) for s in batches]
    for s, ref in zip(batches, want):
        assert all(torch.equal(a, b) for a, b in zip(step(s, False), ref))
    sides = [torch.cuda.Stream() for _ in range(2)]
    static, graphs, got = [], [], []
    for side in sides:
        static.append({k: v.clone() for k, v in batches[0].items()})
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(static[-1], False)
        torch.cuda.current_stream().wait_stream(side)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(step(static[-1], False))
    torch.cuda.synchronize()
    for first in range(4):
        for i, side in enumerate(sides):
            with torch.cuda.stream(side):
                for k, v in batches[(first + i) % 4].items():
                    static[i][k].copy_(v)
                graphs[i].replay()
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(got[i], want[(first + i) % 4]))
    assert nf4.nf4_poll_device_status() == 0


def test_backward_in_a_graph():
    """Forward and backward of the joined block captured and replayed on new inputs."""
    gate, up, down = FP8GatedMLP(*weights(out=528)).quantized_weights()

    def grads(x, s, nw):
        h, y = norm_fp8_gated_mlp(x, nw, gate, up, down, residual=s)
        return torch.autograd.grad((h.square().sum() + y.float().square().sum()), [x, s, nw])

    batches = [(rand(40, 528, seed=k, dtype=BF16), rand(40, 528, seed=k + 1), 1 + rand(528, seed=k + 2, std=0.1))
               for k in (1, 11)]
    want = [grads(*(t.clone().requires_grad_() for t in b)) for b in batches]
    static = [t.clone().requires_grad_() for t in batches[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        grads(*static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = grads(*static)
    for b, ref in zip(batches, want):
        with torch.no_grad():
            for t, v in zip(static, b):
                t.copy_(v)
        graph.replay()
        assert all(torch.equal(a, c) for a, c in zip(got, ref))


@pytest.mark.parametrize("red", [128, 512])
@pytest.mark.parametrize("M", [8, 30, 60, 100, 700])
@pytest.mark.parametrize("dx", [False, True], ids=["fwd", "dx"])
def test_abort_path(M, red, dx):
    """A short limit on a wait that completes anyway: the site is reported, what runs
    on the same SMs next comes out right, and so does the next call."""
    cols = 2048
    shape = (red // 2, cols) if dx else (cols, red)
    wg, wu = (nf4.nf4_fp8_quantize(rand(*shape, seed=i, std=0.02), block_rows=128) for i in (1, 2))
    a, b = (nf4.nf4_fp8_quantize(rand(M, red // 2 if dx else red, seed=i)) for i in (3, 4))
    fn = (lambda: nf4.nf4_fp8_gated_bwd_dx(a, b, wg, wu)) if dx else (lambda: nf4.nf4_fp8_gated_fwd(a, wg, wu)[0])
    bits = lambda t: torch.cat([t.codes.view(torch.uint8).flatten(), t.scale.view(torch.uint8).flatten()]) \
        if isinstance(t, nf4.FP8Tensor) else t                               # noqa: E731
    want = bits(fn())
    assert nf4.nf4_poll_device_status_site() == (0, 0)
    x = rand(300, 512, seed=5)
    for _ in range(4):
        nf4.nf4_set_mma_wait_limit(200)
        try:
            fn()
            after = nf4.nf4_fp8_quantize(x)
            status, site = nf4.nf4_poll_device_status_site()
        finally:
            nf4.nf4_set_mma_wait_limit(0)
        assert status == 7 and (site & 0xffffffff) >> 28 == (7 if dx else 6) and (site >> 24) & 15 == 2
        assert torch.equal(bits(after), bits(nf4.nf4_fp8_quantize(x)))
        assert torch.equal(bits(fn()), want) and nf4.nf4_poll_device_status_site() == (0, 0)


def test_written_outputs_count_as_modified():
    W, X = rand(128, 256), rand(3, 256, dtype=BF16)
    q = nf4.nf4_int4_quantize(W)
    w8, d8 = nf4.nf4_fp8_quantize(W, block_rows=128), nf4.nf4_fp8_quantize(rand(3, 128))
    y, v, x = torch.zeros(3, 128, device=DEV), torch.zeros(128, 256, device=DEV), torch.zeros(3, 256, device=DEV)
    for tensors, call in (([q.codes, q.scale, q.zero], lambda: nf4.nf4_int4_quantize(W, out=q)),
                          ([v], lambda: nf4.nf4_int4_dequantize(q, out=v)),
                          ([y], lambda: nf4.nf4_int4_matmul_fwd(X, q, out=y)),
                          ([x], lambda: nf4.nf4_fp8_gated_bwd_dx(d8, d8, w8, w8, out=x, accumulate=True))):
        before = [t._version for t in tensors]
        call()
        assert all(t._version > b for t, b in zip(tensors, before))
    none = nf4.nf4_int4_quantize(W, zero_point=False)
    assert nf4.nf4_int4_quantize(W, zero_point=False, out=none) is none


def test_operands_off_the_16_byte_grid_are_named():
    w = nf4.nf4_int4_quantize(rand(8, 128))
    x = rand(1 + 128, dtype=BF16)[1:].view(1, 128)
    with pytest.raises(ValueError, match="^X must start on a 16-byte boundary"):
        nf4.nf4_int4_matmul_fwd(x, w)
    with pytest.raises(ValueError, match="^X must start on a 16-byte boundary"):
        nf4.nf4_int4_gated_fwd(x, w, w)
    with pytest.raises(ValueError, match="^W must start on a 16-byte boundary"):
        nf4.nf4_int4_quantize(rand(1 + 128)[1:].view(1, 128))
    codes = torch.zeros(8 * 64 + 1, dtype=torch.uint8, device=DEV)[1:].view(8, 64)
    with pytest.raises(ValueError, match="^w.codes must start on a 16-byte boundary"):
        nf4.nf4_int4_dequantize(nf4.Int4Weight(codes, w.scale, w.zero))
    g = rand(1 + 32, dtype=BF16)
    with pytest.raises(ValueError, match="^u must start on a 16-byte boundary"):
        nf4.nf4_fp8_gated_bwd(g[:32].view(1, 32), g[:32].view(1, 32), g[1:].view(1, 32))
