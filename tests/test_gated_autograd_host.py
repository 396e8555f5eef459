"""The gated block's autograd wrappers on CPU tensors, with the library's calls
replaced by their formulas in torch (nothing rounded to 8 bits): the gradients
are those that torch's own autograd takes of the same block, in every shape and
type, also behind the norm; what second order, a checkpoint and a frozen input do."""
import types

import pytest
import torch
import torch.utils.checkpoint

from dequant_gemm_gb300 import autograd as ag
from tests.test_autograd_host import norm_bwd, norm_fwd

F64 = torch.float64


def act(g, name):
    return torch.nn.functional.silu(g) if name == "silu" else torch.nn.functional.gelu(g, approximate="tanh")


@pytest.fixture
def calls(monkeypatch):
    """The library's calls as formulas; a weight is a namespace with its dense values.
    Returns how often each ran."""
    count = {}

    def counted(name, fn):
        def run(*args, **kw):
            count[name] = count.get(name, 0) + 1
            with torch.no_grad():
                return fn(*args, **kw)
        monkeypatch.setattr(ag, name, run)

    def fwd(x, w, out_dtype=torch.float32):
        return (x.to(F64) @ w.dense.t()).to(out_dtype)

    def dx(dy, w, out_dtype=torch.float32):
        return (dy.to(F64) @ w.dense).to(out_dtype)

    def gated(x, gate, up, activation="silu", save=False):
        g, u = x.to(F64) @ gate.dense.t(), x.to(F64) @ up.dense.t()
        return act(g, activation) * u, *((g, u) if save else (None, None))

    def gated_bwd(dy, g, u, activation="silu"):
        with torch.enable_grad():
            g, u = g.clone().requires_grad_(), u.clone().requires_grad_()
            return torch.autograd.grad(act(g, activation) * u, [g, u], dy.to(F64))

    def gated_dx(dg, du, gate, up, out_dtype=torch.float32):
        return (dg @ gate.dense + du @ up.dense).to(out_dtype)

    counted("nf4_fp8_quantize", lambda x, block_rows=1: x)
    counted("nf4_fp8_matmul_fwd", fwd)
    counted("nf4_fp8_matmul_bwd_dx", dx)
    counted("nf4_fp8_gated_fwd", gated)
    counted("nf4_fp8_gated_bwd", gated_bwd)
    counted("nf4_fp8_gated_bwd_dx", gated_dx)
    counted("nf4_rmsnorm_fwd", lambda x, w, r=None, **kw: norm_fwd(x, w, r, **{**kw, "out_dtype": torch.float32}))
    counted("nf4_rmsnorm_bwd", norm_bwd)
    return count


def rand(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def weights():
    return [types.SimpleNamespace(rows=r, cols=c, dense=rand(r, c, seed=s, dtype=F64) * 0.3)
            for r, c, s in ((24, 16, 1), (24, 16, 2), (32, 24, 3))]


def block(x, name):
    gate, up, down = (w.dense for w in weights())
    return (act(x @ gate.t(), name) * (x @ up.t())) @ down.t()


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lead", [(), (5,), (2, 3)])
def test_block(calls, lead, dtype, name):
    """The sums are fp64; the wrappers round y, the gradient's way through `da` and dx:
    three roundings to the types that they hold them in."""
    x = rand(*lead, 16, seed=4, dtype=dtype).requires_grad_()
    gy = rand(*lead, 32, seed=5)
    y = ag.fp8_gated_mlp(x, *weights(), name, torch.float32)
    X = x.detach().to(F64).requires_grad_()
    Y = block(X, name)
    assert y.shape == Y.shape and torch.allclose(y.to(F64), Y, rtol=2.0 ** -23, atol=1e-30)
    y.backward(gy)
    Y.backward(gy.to(F64))
    u = torch.finfo(dtype).eps / 2
    scale = float(X.grad.abs().max())
    assert x.grad.dtype == dtype and x.grad.shape == x.shape
    # da is rounded where x is bf16 (to bf16), its errors summed over 24 terms
    loose = (24 if dtype == torch.bfloat16 else 0) * 2.0 ** -8 * 3 * scale + 1e-6 * scale
    assert ((x.grad.to(F64) - X.grad).abs() <= 2 * u * X.grad.abs() + loose).all()


@pytest.mark.parametrize("residual", [None, "same", "flat"])
def test_block_behind_the_norm(calls, residual):
    x, nw = rand(2, 3, 16, seed=4).requires_grad_(), (1 + 0.1 * rand(16, seed=5)).requires_grad_()
    r = None if residual is None else rand(*((6, 16) if residual == "flat" else (2, 3, 16)), seed=6).requires_grad_()
    h, y = ag.norm_fp8_gated_mlp(x, nw, *weights(), residual=r, out_dtype=torch.float32)
    gh, gy = rand(2, 3, 16, seed=7), rand(2, 3, 32, seed=8)
    of = [x, nw] + ([] if r is None else [r])
    got = torch.autograd.grad([h, y], of, [gh, gy])
    X, W, R = (None if t is None else t.detach().to(F64).requires_grad_() for t in (x, nw, r))
    H = X if R is None else X + R.reshape(X.shape)
    N = H * torch.rsqrt(H.square().mean(-1, keepdim=True) + 1e-6) * W
    want = torch.autograd.grad([H, block(N, "silu")], [X, W] + ([] if R is None else [R]), [gh.to(F64), gy.to(F64)])
    for a, b, t in zip(got, want, of):
        assert a.shape == t.shape and torch.allclose(a.to(F64), b, rtol=1e-4, atol=1e-5 * float(b.abs().max()))


def test_what_is_not_needed_is_not_done(calls):
    x, nw = rand(5, 16, seed=4), torch.ones(16)
    assert not ag.fp8_gated_mlp(x, *weights()).requires_grad
    x.requires_grad_()
    h, y = ag.norm_fp8_gated_mlp(x, nw, *weights())
    h.sum().backward()                                   # y takes no part
    assert "nf4_fp8_gated_bwd" not in calls and torch.equal(x.grad, torch.ones_like(x))


@pytest.mark.parametrize("joined", [False, True])
def test_second_order_is_refused(calls, joined):
    x, nw = rand(5, 16, seed=4).requires_grad_(), rand(16, seed=5).requires_grad_()

    def loss():
        y = ag.norm_fp8_gated_mlp(x, nw, *weights(), out_dtype=torch.float32)[1] if joined else \
            ag.fp8_gated_mlp(x, *weights(), out_dtype=torch.float32)
        return y.sum() + x.pow(3).sum()                  # a constant gradient reaches y

    of = [x, nw] if joined else [x]
    first = torch.autograd.grad(loss(), of)
    graph = torch.autograd.grad(loss(), of, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(first, graph))
    for g in graph:
        with pytest.raises(RuntimeError, match="once"):
            torch.autograd.grad(g.square().sum(), of, allow_unused=True, retain_graph=True)


def test_checkpointed(calls):
    x = rand(5, 16, seed=4).requires_grad_()
    want, = torch.autograd.grad(ag.fp8_gated_mlp(x, *weights()).float().sum(), x)
    y = torch.utils.checkpoint.checkpoint(lambda x: ag.fp8_gated_mlp(x, *weights()), x, use_reentrant=False)
    assert torch.equal(torch.autograd.grad(y.float().sum(), x)[0], want)


def test_nothing_is_kept_where_no_graph_is_recorded(calls, monkeypatch):
    """Under no_grad and inference_mode a parameter still requires a gradient, and so
    may an input: the projections are not asked for all the same. A checkpoint that
    runs its first pass under no_grad asks for them in the second alone."""
    saves, fwd = [], ag.nf4_fp8_gated_fwd

    def recorded(*args, save=False, **kw):
        saves.append(save)
        return fwd(*args, save=save, **kw)

    monkeypatch.setattr(ag, "nf4_fp8_gated_fwd", recorded)
    x, nw = rand(5, 16, seed=4).requires_grad_(), torch.nn.Parameter(rand(16, seed=5))
    w, r = weights(), rand(5, 16, seed=6)

    def forms(x):
        return [lambda: ag.fp8_gated_mlp(x, *w), lambda: ag.norm_fp8_gated_mlp(x, nw, *w)[1],
                lambda: ag.norm_fp8_gated_mlp(x, nw, *w, residual=r)[1]]

    want = [f() for f in forms(x)]
    assert saves == [True] * 3 and all(y.requires_grad for y in want)
    for mode in (torch.no_grad, torch.inference_mode):
        for leaf in (x, x.detach()):
            saves.clear()
            with mode():
                got = [f() for f in forms(leaf)]
            assert saves == [False] * 3
            assert all(torch.equal(a, b) and not a.requires_grad for a, b in zip(got, want))
    for f in forms(x):
        saves.clear()
        y = torch.utils.checkpoint.checkpoint(lambda _: f(), x, use_reentrant=True)
        assert saves == [False]
        y.float().sum().backward()
        assert saves == [False, True]
    with torch.no_grad():                                # and a graph that is recorded inside
        saves.clear()
        with torch.enable_grad():
            assert ag.fp8_gated_mlp(x, *w).requires_grad and saves == [True]


def test_the_input_is_not_kept(calls):
    """The gradient takes the two projections alone: nothing of the input's size is
    saved, it may change in place before the backward pass (a residual added to it),
    and a second order is refused all the same."""
    seen, w = [], weights()
    leaf, gy = rand(5, 16, seed=4).requires_grad_(), rand(5, 32, seed=7)
    down = types.SimpleNamespace(rows=16, cols=24, dense=rand(16, 24, seed=3, dtype=F64))
    with torch.autograd.graph.saved_tensors_hooks(lambda t: seen.append(t) or t, lambda t: t):
        y = ag.fp8_gated_mlp(leaf * 1.0, *w)             # (the product's factor is no tensor)
    assert sum(t.numel() for t in seen) == 2 * 5 * 24 and all(t.dtype == F64 for t in seen)
    y.float().backward(gy)
    kept = leaf.grad.clone()
    leaf.grad = None
    ag.fp8_gated_mlp(leaf, *w).float().backward(gy)
    assert torch.equal(leaf.grad, kept)

    def step(inplace):
        h = leaf * 1.0
        y = ag.fp8_gated_mlp(h, w[0], w[1], down, "silu", torch.float32)
        if inplace:
            h += y
        else:
            h = h + y
        return h

    g = rand(5, 16, seed=8)
    want, = torch.autograd.grad(step(False), leaf, g)
    got, = torch.autograd.grad(step(True), leaf, g)
    assert torch.equal(got, want)
    once, = torch.autograd.grad(step(True), leaf, g, create_graph=True)
    assert torch.equal(once, want)
    with pytest.raises(RuntimeError, match="once"):
        torch.autograd.grad(once.square().sum(), leaf)


def test_no_gradient_is_zeros(calls):
    """Where nothing comes back for y, x gets zeros and no kernel runs."""
    class Cut(torch.autograd.Function):
        @staticmethod
        def forward(ctx, y):
            return y.clone()

        @staticmethod
        def backward(ctx, gy):
            return None

    x = rand(2, 3, 16, seed=4, dtype=torch.bfloat16).requires_grad_()
    Cut.apply(ag.fp8_gated_mlp(x, *weights())).float().sum().backward()
    assert torch.equal(x.grad, torch.zeros_like(x)) and "nf4_fp8_gated_bwd" not in calls
