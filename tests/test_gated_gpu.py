"""The gated block on 8-bit operands against 64 bits.

G and U are products of 8-bit operands, with their bound
  e = (128 * 2^-23 + (3 + blocks) * 2^-24) * sum of |products|
(tests/test_fp8_gpu.py). sigma(p) carries six roundings of its exponent, which
count |p| each where sigma is small (p < 0; for p > 0, p exp(-p) < 0.4), the
exponential's 2^-22, the sum's 2^-24 and the reciprocal's 2^-23: with the two
products, act(g) u is off by r = (6 max(0, -p) + 12) * 2^-24 of itself, and by
2^-126 |g u| where exp(-p) leaves fp32. |act'| < 1.13. So
  |Y - Y_ref| <= |u| 1.13 eG + (|act| + 1.13 eG) eU + r |act u| + 2^-126 |g u|.
A 16-bit output adds half an ulp. An 8-bit one is its code times the block's
scale: half a step is 2^-4 of a normal code's value and 2^-10 of a scale below,
and scaling rounds three times in fp32."""
import pytest
import torch

import dequant_gemm_gb300 as nf4
from oracle import fp8_oracle as o8
from oracle import gated_oracle as o

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8, F32, BF16 = torch.float8_e4m3fn, torch.float32, torch.bfloat16
U24 = 2.0 ** -24


def make(rows, cols, seed, std=1.0, dtype=F32):
    g = torch.Generator(device="cpu").manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * std
    x[:, torch.randint(0, cols, (max(1, cols // 200),), generator=g)] *= 10
    return x.to(dtype).to(DEV)


def weights(N, K, seed=5):
    return [nf4.nf4_fp8_quantize(make(N, K, seed + i, 0.02), block_rows=128) for i in (0, 1)]


def values64(q):
    table = torch.from_numpy(o8.VALUES).to(DEV)
    s = q.scale.double().repeat_interleave(q.block_rows, 0)[:q.rows]
    return table[q.codes.view(torch.uint8).long()] * s.repeat_interleave(128, 1)[:, :q.cols]


def on_gpu(f, x, name):
    return [torch.from_numpy(t).to(DEV) for t in f(x.cpu().numpy(), name)]


def project(a, w):
    """(product, its bound)."""
    A, W = values64(a), values64(w).t()
    blocks = -(-a.cols // 128)
    return A @ W, (128 * 2.0 ** -23 + (3 + blocks) * U24) * (A.abs() @ W.abs())


def relative(g, name):
    p, _ = on_gpu(o.exponent, g, name)
    return (6 * (-p).clamp(min=0) + 12) * U24


def reference(x, wg, wu, name):
    """(G, eG), (U, eU), (Y, eY)."""
    (g, eg), (u, eu) = project(x, wg), project(x, wu)
    f, _ = on_gpu(o.act, g, name)
    e = u.abs() * 1.13 * eg + (f.abs() + 1.13 * eg) * eu + relative(g, name) * 1.01 * (f * u).abs() \
        + 2.0 ** -126 * (g * u).abs() + 1e-44
    return (g, eg), (u, eu), (f * u, e)


FMAX = 2.0 ** 128 * (1 - 2.0 ** -25)     # rounds to an infinity in fp32 (bf16's is further out by 2^-9)


def assert_near(got, want, bound):
    """Within `bound`; a value past fp32's range is an infinity of its sign, one
    whose bound reaches past it may be."""
    past = want.abs() - bound >= FMAX
    assert torch.equal(got.double()[past], want[past].sign() * float("inf"))
    bad = ~((got.double() - want).abs() <= bound) & (want.abs() + bound < FMAX)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, first {bad.nonzero()[0].tolist()}"


def assert_block_scaled(q, want, bound):
    """Codes and scales of a tensor that is known to `bound`."""
    rows, cols = want.shape
    pad = lambda t: torch.nn.functional.pad(t, (0, -cols % 128)).reshape(rows, -1, 128)  # noqa: E731
    amax, e = pad(want.abs()).amax(2), pad(bound).amax(2)
    past = amax - e >= FMAX                # an infinity makes its block NaN
    sure = (amax + e < FMAX)
    assert (~q.scale[past].isfinite()).all() and pad(values64(q))[past].isnan().any(1).all()
    want = torch.where(sure.repeat_interleave(128, 1)[:, :cols], want, 0.0)
    q = nf4.FP8Tensor(torch.where(sure.repeat_interleave(128, 1)[:, :cols], q.codes.float(), 0.0).to(F8),
                      torch.where(sure, q.scale, 0.0))
    amax, e = pad(want.abs()).amax(2), pad(bound).amax(2)
    assert ((q.scale.double() * 448 - amax).abs() <= e + 2.0 ** -22 * amax + 2.0 ** -117).all()
    s = q.scale.double().repeat_interleave(128, 1)[:, :cols]
    assert_near(values64(q), want, torch.maximum(want.abs() * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -20)
                + 1.07 * bound + 2.0 ** -117)


def check_forward(x, wg, wu, name, outs=(F8, BF16, F32), save=(False, True)):
    ref_g, ref_u, (y, e) = reference(x, wg, wu, name)
    for out in outs:
        for keep in save:
            got, g, u = nf4.nf4_fp8_gated_fwd(x, wg, wu, activation=name, out_dtype=out, save=keep)
            if out == F8:
                assert_block_scaled(got, y, e)
            else:
                assert got.dtype == out
                assert_near(got, y, e * (1 + 2.0 ** -8) + (2.0 ** -8 * y.abs() if out == BF16 else U24 * y.abs()))
            assert (g is None) == (u is None) == (not keep)
            if keep:
                for t, (r, er) in ((g, ref_g), (u, ref_u)):
                    assert t.dtype == BF16
                    assert_near(t, r, er * (1 + 2.0 ** -8) + 2.0 ** -8 * r.abs())
            again = nf4.nf4_fp8_gated_fwd(x, wg, wu, activation=name, out_dtype=out, save=keep)
            for a, b in zip((got, g, u), again):
                if isinstance(a, nf4.FP8Tensor):
                    assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8))
                    assert torch.equal(a.scale, b.scale)
                elif a is not None:
                    assert torch.equal(a, b)
    assert nf4.nf4_poll_device_status() == 0


SHAPES = [(1, 16, 16), (2, 144, 272), (5, 1040, 528), (16, 272, 1040), (17, 256, 128), (33, 400, 400),
          (64, 528, 2064), (65, 128, 144), (100, 640, 640), (128, 272, 272), (129, 400, 528), (250, 512, 896),
          (300, 1040, 1552), (513, 2064, 1040), (1000, 784, 3600), (1, 3584, 4096), (8, 128, 8192),
          (600, 16, 16)]


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M, N, K", SHAPES)
def test_forward(M, N, K, name):
    x = nf4.nf4_fp8_quantize(make(M, K, M + N))
    wg, wu = weights(N, K)
    check_forward(x, wg, wu, name)


@pytest.mark.parametrize("M", [3, 40, 150, 300])
def test_one_hot_rows_return_the_weights(M):
    """One code of 1.0 a row: G and U are one weight value each, exact up to the
    scales' roundings; every column of both weights."""
    N, K = 272, 400
    wg, wu = weights(N, K)
    codes = torch.zeros(M, K, device=DEV)
    at = (torch.arange(M, device=DEV) * 7) % K
    codes[torch.arange(M, device=DEV), at] = 1.0
    x = nf4.FP8Tensor(codes.to(F8), torch.rand(M, 4, device=DEV) * 30 + 0.5)
    y, g, u = nf4.nf4_fp8_gated_fwd(x, wg, wu, out_dtype=F32, save=True)
    s = x.scale.double()[torch.arange(M, device=DEV), at // 128][:, None]
    G, U = values64(wg).t()[at] * s, values64(wu).t()[at] * s
    for t, r in ((g, G), (u, U)):
        assert_near(t, r, (2.0 ** -8 + 4 * U24) * r.abs())
    f, slope = on_gpu(o.act, G, "silu")
    assert_near(y, f * U, (relative(G, "silu") + 4 * U24) * (f * U).abs() + 3 * U24 * (slope * G * U).abs())


@pytest.mark.parametrize("M", [4, 50, 140, 290])
def test_nan_and_zero_rows_stay_in_their_rows(M):
    wg, wu = weights(272, 400)
    x = make(M, 400, 6)
    x[1, 300], x[2] = float("nan"), 0.0
    y, g, u = nf4.nf4_fp8_gated_fwd(nf4.nf4_fp8_quantize(x), wg, wu, save=True)
    v = nf4.nf4_fp8_dequantize(y)
    assert v[1].isnan().all() and g[1].isnan().all() and (v[2] == 0).all() and (y.scale[2] == 0).all()
    assert not v[0].isnan().any() and not v[3:].isnan().any()


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M", [5, 300])
def test_activation_far_out(M, name):
    """Projections from 1e-30 to 1e30: scales of hand-made operands."""
    K, N = 144, 128
    wg, wu = weights(N, K)
    x = nf4.nf4_fp8_quantize(make(M, K, 3))
    x.scale.mul_(10.0 ** torch.linspace(-30, 29, M, device=DEV)[:, None])
    check_forward(x, wg, wu, name, outs=(F32, F8) if M == 300 else (F32, BF16))


def test_empty_calls():
    wg, wu = weights(32, 256)
    for out in (F8, F32):
        y, g, u = nf4.nf4_fp8_gated_fwd(nf4.alloc_fp8(0, 256, DEV), wg, wu, out_dtype=out, save=True)
        assert (y.codes if out == F8 else y).shape == (0, 32) and g.shape == u.shape == (0, 32)
        none = nf4.alloc_fp8(0, 256, DEV, 128)
        y, _, _ = nf4.nf4_fp8_gated_fwd(nf4.alloc_fp8(3, 256, DEV), none, none, out_dtype=out)
        assert (y.codes if out == F8 else y).shape == (3, 0)
        thin = nf4.alloc_fp8(32, 0, DEV, 128)
        y, g, u = nf4.nf4_fp8_gated_fwd(nf4.alloc_fp8(3, 0, DEV), thin, thin, out_dtype=out, save=True)
        v = nf4.nf4_fp8_dequantize(y) if out == F8 else y
        assert (v == 0).all() and (g == 0).all() and (u == 0).all()
    dg, du = nf4.nf4_fp8_gated_bwd(*(torch.empty(0, 32, device=DEV, dtype=t) for t in (F32, BF16, BF16)))
    assert dg.rows == du.rows == 0
    dx = nf4.nf4_fp8_gated_bwd_dx(nf4.alloc_fp8(3, 0, DEV), nf4.alloc_fp8(3, 0, DEV), none, none)
    assert dx.shape == (3, 256) and (dx == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16, torch.float16])
@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M, N", [(1, 16), (3, 144), (130, 1040), (257, 256)])
def test_gradients_of_the_product(M, N, name, dtype):
    """dG = dY U act'(G): act' = s + g s (1 - s) p', with s off by r (above), 1 - s
    by r s + 2^-24, five more roundings of either term, and three of the product
    with dY and U."""
    g = torch.Generator(device="cpu").manual_seed(M)
    G = (torch.randn(M, N, generator=g) * 4).bfloat16().to(DEV)
    U = torch.randn(M, N, generator=g).bfloat16().to(DEV)
    dy = (torch.randn(M, N, generator=g) * 0.01).to(dtype).to(DEV)
    G[0, 0], G[0, 3], U[0, 5] = -60.0, 90.0, 0.0
    if M > 2:
        dy[1] = 0.0
        G[2, 7:9] = torch.tensor([1e20, -1e20])
    dg, du = nf4.nf4_fp8_gated_bwd(dy, G, U, activation=name)
    d, gd, ud = dy.double(), G.double(), U.double()
    (f, slope), (p, dp) = on_gpu(o.act, gd, name), on_gpu(o.exponent, gd, name)
    s, r = torch.sigmoid(p), (6 * (-p).clamp(min=0) + 12) * U24
    near = gd.abs() <= 1e10                 # beyond, s (1 - s) is 0 and p' may be infinite in the reference
    f, slope = torch.where(near, f, gd.clamp(min=0)), torch.where(near, slope, (gd > 0).double())
    curve = torch.where(near, (gd * dp).abs(), 0.0)
    e = r * s + curve * (r * s * (1 - s) + s * (r * s + U24)) + 8 * U24 * (s + curve * s * (1 - s)) + 2.0 ** -126 * (1 + curve)
    # far out on the positive side 1 - s is a rounded 0, on the negative s is
    assert_block_scaled(dg, d * ud * slope, (d * ud).abs() * e * 1.01 + 3 * U24 * (d * ud * slope).abs() + 1e-44)
    assert_block_scaled(du, d * f, d.abs() * (r * f.abs() * 1.01 + 2.0 ** -126 * gd.abs().clamp(max=1e10)) + 1e-44)
    again = nf4.nf4_fp8_gated_bwd(dy, G, U, activation=name)
    for a, b in zip((dg, du), again):
        assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8)) and torch.equal(a.scale, b.scale)


@pytest.mark.parametrize("M, N, K", SHAPES)
def test_input_gradient(M, N, K):
    """The products' bound over both reductions, one after the other."""
    dg, du = (nf4.nf4_fp8_quantize(make(M, N, M + N + i, 0.1)) for i in (0, 1))
    wg, wu = weights(N, K)
    pairs = [(values64(d), values64(w)) for d, w in ((dg, wg), (du, wu))]
    ref = sum(a @ b for a, b in pairs)
    terms = sum(a.abs() @ b.abs() for a, b in pairs)
    bound = (128 * 2.0 ** -23 + (3 + 2 * -(-N // 128)) * U24) * terms
    for dt in (F32, BF16):
        u = 2.0 ** -8 if dt == BF16 else U24
        dx = nf4.nf4_fp8_gated_bwd_dx(dg, du, wg, wu, out_dtype=dt)
        assert_near(dx, ref, bound * (1 + u) + u * ref.abs())
        assert torch.equal(dx, nf4.nf4_fp8_gated_bwd_dx(dg, du, wg, wu, out_dtype=dt))
        out = make(M, K, 9).to(dt)
        before = out.double()
        assert nf4.nf4_fp8_gated_bwd_dx(dg, du, wg, wu, out=out, accumulate=True) is out
        total = ref + before
        assert_near(out, total, (bound + U24 * (total.abs() + before.abs())) * (1 + u) + u * total.abs())
    assert nf4.nf4_poll_device_status() == 0


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
def test_gradients_against_differences(name):
    """The derivative of sum(Y * c) along a direction of X, by central differences
    of the 64-bit definition at the 8-bit operands' values, against <dX, v>:
    dX's error is its 8-bit factors' (2^-4 of each dG and dU value, 2^-8 for the
    bf16 G and U that they are taken from) and the products' own."""
    M, N, K = 12, 272, 400
    x = nf4.nf4_fp8_quantize(make(M, K, 1))
    wg, wu = weights(N, K)
    X, Wg, Wu = values64(x), values64(wg), values64(wu)
    c = make(M, N, 7, 0.1)
    v = make(M, K, 8).double()

    def total(t):
        G, U = (X + t * v) @ Wg.t(), (X + t * v) @ Wu.t()
        return float((on_gpu(o.act, G, name)[0] * U * c.double()).sum())

    h = 1e-5
    want = (total(h) - total(-h)) / (2 * h)
    _, g, u = nf4.nf4_fp8_gated_fwd(x, wg, wu, activation=name, save=True)
    dg, du = nf4.nf4_fp8_gated_bwd(c, g, u, activation=name)
    got = float((nf4.nf4_fp8_gated_bwd_dx(dg, du, wg, wu).double() * v).sum())
    # each dG, dU value within 2^-4 of itself or 2^-10 of its scale, plus what the
    # rounded G and U move it by (|act''| < 1.2, |act'| < 1.13)
    G, U, C = X @ Wg.t(), X @ Wu.t(), c.double().abs()
    f, slope = on_gpu(o.act, G, name)
    moved = 2.0 ** -8 * 1.01
    eg = C * (U.abs() * 1.2 * moved * G.abs() + moved * (U * slope).abs() + 1.4 * moved ** 2 * (G * U).abs())
    eu = C * 1.13 * moved * G.abs()
    eight = lambda q, t: torch.maximum(t.abs() * 2.0 ** -4, q.scale.double().repeat_interleave(128, 1)[:, :N] * 2.0 ** -10) * 1.1  # noqa: E731
    eg = eg + eight(dg, C * U * slope) + 0.07 * eg
    eu = eu + eight(du, C * f) + 0.07 * eu
    # the errors are independent of v's signs: bounded term by term
    bound = float((eg * (v @ Wg.t()).abs()).sum() + (eu * (v @ Wu.t()).abs()).sum())
    assert abs(got - want) <= bound + 1e-3 * abs(want)


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
def test_gradients_along_themselves(name):
    """The derivative of sum(Y * c) along the 64-bit gradient v itself, by central
    differences, against <dX, v>: no cancellation hides a lost part, since each of
    both reductions makes up more than twice the bound.
    G and U are off by their products' e and bf16's 2^-8 (moved); |act''| < 0.81, so
    dG = c U act'(G) is off by |c| (0.81 |U| moved(G) + |act'| moved(U) + the product of
    both), dU = c act(G) by 1.13 |c| moved(G), the arithmetic of either by 2^-12 of its
    terms (|p| < 160: r < 2^-14, above). In 8 bits 2^-4 of the value or 2^-10 of the
    scale, three roundings in fp32. Then the input gradient's own bound."""
    M, N, K = 12, 272, 2048
    x = nf4.nf4_fp8_quantize(make(M, K, 1))
    wg, wu = weights(N, K)
    X, Wg, Wu = values64(x), values64(wg), values64(wu)
    (G, eG), (U, eU) = project(x, wg), project(x, wu)
    c = make(M, N, 7, 0.1)
    C = c.double()
    f, slope = on_gpu(o.act, G, name)
    p, dp = on_gpu(o.exponent, G, name)
    assert float(p.abs().max()) < 160
    tG, tU = C * U * slope, C * f
    v = tG @ Wg + tU @ Wu
    v *= M * K / float(v.abs().sum())
    parts = float((tG * (v @ Wg.t())).sum()), float((tU * (v @ Wu.t())).sum())

    def total(t):
        A, B = (X + t * v) @ Wg.t(), (X + t * v) @ Wu.t()
        return float((on_gpu(o.act, A, name)[0] * B * C).sum())

    h = 1e-5
    want = (total(h) - total(-h)) / (2 * h)
    assert abs(want - sum(parts)) <= 1e-6 * abs(want)     # the formulas' own gradient
    _, g, u = nf4.nf4_fp8_gated_fwd(x, wg, wu, activation=name, save=True)
    dg, du = nf4.nf4_fp8_gated_bwd(c, g, u, activation=name)
    got = float((nf4.nf4_fp8_gated_bwd_dx(dg, du, wg, wu).double() * v).sum())
    mG, mU = (e + 2.0 ** -8 * (t.abs() + e) for t, e in ((G, eG), (U, eU)))
    each = 2.0 ** -12 * C.abs() * (1 + (G * dp).abs())
    bG = C.abs() * (0.81 * U.abs() * mG + slope.abs() * mU + 0.81 * mG * mU) + each * (U.abs() + mU)
    bU = 1.13 * C.abs() * mG + each * G.abs()

    def eight(q, t, b):
        s = q.scale.double().repeat_interleave(128, 1)[:, :N]
        return b + torch.maximum((t.abs() + b) * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -20)

    bG, bU = eight(dg, tG, bG), eight(du, tU, bU)
    terms = (tG.abs() + bG) @ Wg.abs() + (tU.abs() + bU) @ Wu.abs()
    own = (128 * 2.0 ** -23 + (4 + 2 * -(-N // 128)) * U24) * float((terms * v.abs()).sum())
    bound = float((bG * (v @ Wg.t()).abs()).sum() + (bU * (v @ Wu.t()).abs()).sum()) + own + 1e-6 * abs(want)
    assert all(q > 2 * bound for q in parts)
    assert abs(got - want) <= bound


def test_row_slices_and_another_stream():
    wg, wu = weights(256, 400)
    q = nf4.nf4_fp8_quantize(make(200, 400, 6))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for lo, hi in ((1, 2), (7, 50), (3, 200)):
            part = nf4.FP8Tensor(q.codes[lo:hi], q.scale[lo:hi])
            check_forward(part, wg, wu, "silu", outs=(BF16, F8), save=(True,))
    side.synchronize()


def test_the_same_weight_twice():
    """gate and up may be one weight: Y = act(G) G."""
    wg, _ = weights(272, 400)
    for M in (7, 300):
        check_forward(nf4.nf4_fp8_quantize(make(M, 400, 2)), wg, wg, "silu", outs=(F32,), save=(True,))


def test_offsets_beyond_32_bits():
    """Outputs of more than 2^31 elements, and inputs: the last rows come out right."""
    M, N, K = 140_000, 16_384, 32
    wg, wu = weights(N, K)
    x = nf4.alloc_fp8(M, K, DEV)
    x.codes.view(torch.uint8).zero_()
    x.scale.fill_(1.0)
    tail = nf4.nf4_fp8_quantize(make(64, K, 8))
    x.codes[-64:], x.scale[-64:] = tail.codes, tail.scale
    y, g, u = nf4.nf4_fp8_gated_fwd(x, wg, wu, save=True)
    want = nf4.nf4_fp8_gated_fwd(nf4.FP8Tensor(x.codes[-300:], x.scale[-300:]), wg, wu, save=True)
    assert torch.equal(y.codes[-300:].view(torch.uint8), want[0].codes.view(torch.uint8))
    assert torch.equal(g[-300:], want[1]) and torch.equal(u[-300:], want[2])
    ref_g, _, (ref, e) = reference(tail, wg, wu, "silu")
    assert_block_scaled(nf4.FP8Tensor(y.codes[-64:], y.scale[-64:]), ref, e)
    assert not y.scale[:-64].any()
    dy = torch.zeros(M, N, dtype=BF16, device=DEV)
    dy[-64:] = make(64, N, 3, dtype=BF16)
    dg, du = nf4.nf4_fp8_gated_bwd(dy, g, u)
    wdg, wdu = nf4.nf4_fp8_gated_bwd(dy[-64:], g[-64:], u[-64:])
    for a, b in ((dg, wdg), (du, wdu)):
        assert torch.equal(a.codes[-64:].view(torch.uint8), b.codes.view(torch.uint8))
        assert torch.equal(a.scale[-64:], b.scale) and not a.scale[:-64].any()
