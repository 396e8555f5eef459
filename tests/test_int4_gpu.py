"""4-bit weights in groups on the GPU against the oracle.

The quantizer's steps are fp32 with one rounding each: codes, scales and zero
points match bit for bit. A product's error bound: (code - zero) x is exact in
fp32; a group's (at most) 128 products are summed with one rounding or
truncation each (2^-23); the scale's product, and the additions of groups and of
a row's parts (at most 48 more), round once each (2^-24). An output rounds once
to its type, and once in fp32 where it is added to what was there. The gated
block: as in tests/test_gated_gpu.py."""
import numpy as np
import pytest
import torch

import dequant_gemm_gb300 as nf4
from oracle import gated_oracle as o
from tests.test_gated_gpu import assert_near, on_gpu, relative

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U24 = 2.0 ** -24
UNIT = {F32: U24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {F32: 0.0, BF16: 0.0, F16: 2.0 ** -25}     # half of fp16's smallest step


def make(rows, cols, seed, std=1.0, dtype=F32):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return (torch.randn(rows, cols, generator=g) * std).to(dtype)


def weight(N, K, group, zero=True, scale=BF16, seed=5):
    return nf4.nf4_int4_quantize(make(N, K, seed, 0.02).to(DEV), group=group, zero_point=zero, scale_dtype=scale)


def values64(w):
    v = o.int4_values(w.codes.cpu().numpy(), w.scale.double().cpu().numpy(),
                      None if w.zero is None else w.zero.cpu().numpy())
    return torch.from_numpy(v).to(DEV)


def product(x, w):
    """(X w^T, its bound) in 64 bits."""
    X, W = x.double(), values64(w).t()
    terms = X.abs() @ W.abs()
    groups = w.cols // w.group
    return X @ W, (w.group * 2.0 ** -23 + (groups + 50) * U24) * terms


@pytest.mark.parametrize("scale", [BF16, F16])
@pytest.mark.parametrize("zero", [True, False])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_quantize_is_bit_exact(dtype, group, zero, scale):
    for rows, cols in ((1, 128), (3, 384), (129, 1152)):
        w = make(rows, cols, rows, 0.02, dtype)
        w[0, :32] = 0
        w[rows // 2, 64:128] = w[rows // 2, 64:128].abs() + 0.01      # one-sided groups
        if dtype != F16:
            w[rows - 1, 0] = 1e4
        q = nf4.nf4_int4_quantize(w.to(DEV), group=group, zero_point=zero, scale_dtype=scale)
        codes, s, z = o.int4_quantize(w.float().numpy(), group, zero, "bf16" if scale == BF16 else "f16")
        assert np.array_equal(q.scale.float().cpu().numpy(), s)
        assert (q.zero is not None) == zero
        if zero:
            assert np.array_equal(q.zero.cpu().numpy(), z)
        assert np.array_equal(q.codes.cpu().numpy(), o.int4_pack(codes))
        for dt in (F32, BF16, F16):
            v = nf4.nf4_int4_dequantize(q, out_dtype=dt)
            assert torch.equal(v, values64(q).float().to(dt))         # (code - zero) * scale is exact in fp32
        out = nf4.Int4Weight(torch.zeros_like(q.codes), torch.zeros_like(q.scale),
                             torch.zeros_like(q.zero) if zero else None)
        assert nf4.nf4_int4_quantize(w.to(DEV), group=group, zero_point=zero, scale_dtype=scale, out=out) is out
        assert torch.equal(out.codes, q.codes) and torch.equal(out.scale, q.scale)


def test_quantize_of_extreme_values():
    """Ties of the quotient, tiny and large groups, subnormal scales."""
    w = torch.zeros(8, 64)
    w[0] = torch.arange(64) / 2.0                   # (hi - lo) / 15 and halves
    w[1] = torch.linspace(-7.5, 7.5, 64)
    w[2] = 1e-38
    w[3, 5], w[3, 40] = 3e36, -3e36
    w[4] = 1e-42
    w[5] = -torch.arange(64).float()
    w[6, 0] = 2.0 ** -130
    w[7] = torch.tensor([0.5, -0.5] * 32)
    for zero in (True, False):
        for group in (32, 64):
            q = nf4.nf4_int4_quantize(w.to(DEV), group=group, zero_point=zero)
            codes, s, z = o.int4_quantize(w.numpy(), group, zero, "bf16")
            assert np.array_equal(q.scale.float().cpu().numpy(), s)
            assert np.array_equal(q.codes.cpu().numpy(), o.int4_pack(codes))
            assert not zero or np.array_equal(q.zero.cpu().numpy(), z)


SHAPES = [(1, 1, 128), (1, 8, 256), (1, 17, 384), (1, 512, 3584), (1, 4096, 4096), (2, 100, 1280), (3, 33, 640), (7, 130, 2176),
          (8, 256, 128), (9, 300, 1152), (15, 31, 4352), (16, 272, 1024), (17, 64, 512), (33, 129, 896),
          (48, 1000, 256), (1, 64, 18944), (5, 48, 53248), (130, 40, 384)]


@pytest.mark.parametrize("M, N, K", SHAPES)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_product(M, N, K, group):
    K += {32: 32, 64: 64, 128: 0}[group]             # rows that end inside a 128-block
    for i, (xt, zero) in enumerate(((BF16, True), (F16, False), (F16, True), (BF16, False))):
        x = make(M, K, M + N, dtype=xt).to(DEV)
        w = weight(N, K, group, zero, (BF16, F16)[(i + M) % 2])
        ref, bound = product(x, w)
        for dt in (F32, BF16, F16):
            y = nf4.nf4_int4_matmul_fwd(x, w, out_dtype=dt)
            assert y.shape == (M, N) and y.dtype == dt
            assert_near(y, ref, bound * (1 + UNIT[dt]) + UNIT[dt] * ref.abs() + TINY[dt])
            assert torch.equal(y, nf4.nf4_int4_matmul_fwd(x, w, out_dtype=dt))
        out = make(M, N, 9).to(F32).to(DEV)
        before = out.double()
        assert nf4.nf4_int4_matmul_fwd(x, w, out=out, accumulate=True) is out
        total = ref + before
        assert_near(out, total, bound + U24 * (2 * total.abs() + before.abs()))


@pytest.mark.parametrize("M, N, K", SHAPES)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_gated(M, N, K, group):
    K += {32: 32, 64: 64, 128: 0}[group]
    for name, xt, zeros in (("silu", BF16, (True, True)), ("gelu_tanh", F16, (False, True))):
        x = make(M, K, M + N, dtype=xt).to(DEV)
        a, b = (weight(N, K, group, z, xt, seed=s) for z, s in zip(zeros, (5, 6)))
        (g, eg), (u, eu) = product(x, a), product(x, b)
        f, _ = on_gpu(o.act, g, name)
        e = u.abs() * 1.13 * eg + (f.abs() + 1.13 * eg) * eu + relative(g, name) * 1.01 * (f * u).abs()
        for dt in (None, F32):
            y = nf4.nf4_int4_gated_fwd(x, a, b, activation=name, out_dtype=dt)
            dt = xt if dt is None else dt
            assert y.dtype == dt
            assert_near(y, f * u, e * (1 + UNIT[dt]) + UNIT[dt] * (f * u).abs() + TINY[dt] + 1e-38)


@pytest.mark.parametrize("M, N, K", [(1, 20, 262144), (3, 40, 262144), (16, 20, 100352), (20, 33, 60000 // 128 * 128),
                                     (1, 40000, 256), (12, 5000, 384), (300, 600, 256)])
def test_longest_rows_and_many_tiles(M, N, K):
    """Fewer tokens a tile where the reduction is long, several row tiles a CTA
    where there are many rows."""
    x = make(M, K, M + N, dtype=BF16).to(DEV)
    a, b = weight(N, K, 128), weight(N, K, 128, seed=6)
    ref, bound = product(x, a)
    assert_near(nf4.nf4_int4_matmul_fwd(x, a), ref, bound + U24 * ref.abs())
    (g, eg), (u, eu) = (ref, bound), product(x, b)
    f, _ = on_gpu(o.act, g, "silu")
    e = u.abs() * 1.13 * eg + (f.abs() + 1.13 * eg) * eu + relative(g, "silu") * 1.01 * (f * u).abs()
    assert_near(nf4.nf4_int4_gated_fwd(x, a, b, out_dtype=F32), f * u, e * (1 + U24) + U24 * (f * u).abs() + 1e-38)


@pytest.mark.parametrize("M", [1, 5, 16, 20])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_one_hot_tokens_return_the_weight(M, group):
    """Every element of the weight once: Y is (code - zero) * scale, exact."""
    N, K = 40, 1152
    w = weight(N, K, group)
    W = values64(w)
    for k0 in range(0, K, M):
        at = torch.arange(k0, k0 + M, device=DEV) % K
        x = torch.zeros(M, K, dtype=BF16, device=DEV)
        x[torch.arange(M, device=DEV), at] = 1.0
        assert torch.equal(nf4.nf4_int4_matmul_fwd(x, w).double(), W.t()[at])


def test_nan_and_infinity_stay_in_their_tokens():
    w = weight(100, 640, 64)
    for M in (4, 20):
        x = make(M, 640, 3, dtype=BF16).to(DEV)
        x[1, 600], x[2, 5] = float("nan"), float("inf")
        y = nf4.nf4_int4_matmul_fwd(x, w)
        assert y[1].isnan().all() and not y[2].isfinite().any()
        assert y[0].isfinite().all() and y[3:].isfinite().all()


def test_activations_of_any_size():
    """bf16 tokens of 1e-30 to 1e30 enter as they are."""
    w = weight(64, 512, 128)
    x = (make(12, 512, 1) * 10.0 ** torch.linspace(-30, 30, 12)[:, None]).bfloat16().to(DEV)
    ref, bound = product(x, w)
    assert_near(nf4.nf4_int4_matmul_fwd(x, w), ref, bound + U24 * ref.abs())


def test_empty_calls():
    w = weight(32, 256, 64)
    assert nf4.nf4_int4_matmul_fwd(torch.empty(0, 256, dtype=BF16, device=DEV), w).shape == (0, 32)
    none = nf4.nf4_int4_quantize(torch.empty(0, 256, device=DEV))
    assert nf4.nf4_int4_matmul_fwd(torch.ones(3, 256, dtype=BF16, device=DEV), none).shape == (3, 0)
    thin = nf4.nf4_int4_quantize(torch.empty(32, 0, device=DEV))
    x = torch.empty(3, 0, dtype=BF16, device=DEV)
    assert (nf4.nf4_int4_matmul_fwd(x, thin) == 0).all() and (nf4.nf4_int4_gated_fwd(x, thin, thin) == 0).all()
    assert nf4.nf4_int4_dequantize(thin).shape == (32, 0)


def test_row_slices_and_another_stream():
    """A run of the weight's rows: scales and zero points that start anywhere."""
    w, x = weight(100, 640, 128), make(3, 640, 2, dtype=BF16).to(DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for lo, hi in ((1, 2), (7, 50), (3, 100)):
            part = nf4.Int4Weight(w.codes[lo:hi], w.scale[lo:hi], w.zero[lo:hi])
            ref, bound = product(x, part)
            assert_near(nf4.nf4_int4_matmul_fwd(x, part), ref, bound + U24 * ref.abs())
            assert torch.equal(nf4.nf4_int4_dequantize(part).double(), values64(part))
    side.synchronize()


def test_offsets_beyond_32_bits():
    """A weight of more than 2^32 values: the last rows come out right."""
    N, K = 262_160, 16_512
    w = nf4.Int4Weight(torch.full((N, K // 2), 0x88, dtype=torch.uint8, device=DEV),
                       torch.zeros(N, K // 128, dtype=BF16, device=DEV))
    tail = weight(40, K, 128, zero=False)
    w.codes[-40:], w.scale[-40:] = tail.codes, tail.scale
    for M in (1, 9):
        x = make(M, K, 2, dtype=BF16).to(DEV)
        y = nf4.nf4_int4_matmul_fwd(x, w)
        ref, bound = product(x, tail)
        assert_near(y[:, -40:], ref, bound + U24 * ref.abs())
        assert not y[:, :-40].any()


@pytest.mark.parametrize("M, N, K", [
    (1, 24, 1056), (1, 1240, 4096), (1, 2888, 4096), (1, 40, 4096), (2, 2928, 4096), (1, 2504, 4096), (2, 64, 3200),
    (1, 16, 6400), (3, 24, 3200), (1, 760, 8192), (1, 16, 12800), (8, 24, 2048), (7, 2464, 2048), (5, 2496, 2048),
    (17, 3664, 1056), (11, 2328, 1056), (100, 648, 3200), (33, 2312, 2048), (17, 936, 3200), (17, 376, 6400),
    (11, 24, 12800), (160, 3872, 32), (160, 3848, 512), (64, 272, 18944), (160, 296, 8192)])
def test_clusters_and_parts(M, N, K):
    """Reductions split over clusters of 1 to 8 and over 1 to 16 warps of a CTA, in
    numbers that divide neither, with one row tile or several."""
    x = make(M, K, M + N, dtype=BF16).to(DEV)
    a, b = weight(N, K, 32), weight(N, K, 32, seed=6)
    (g, eg), (u, eu) = product(x, a), product(x, b)
    y = nf4.nf4_int4_matmul_fwd(x, a)
    assert_near(y, g, eg + U24 * g.abs())
    assert torch.equal(y, nf4.nf4_int4_matmul_fwd(x, a))
    f, _ = on_gpu(o.act, g, "silu")
    e = u.abs() * 1.13 * eg + (f.abs() + 1.13 * eg) * eu + relative(g, "silu") * 1.01 * (f * u).abs()
    y = nf4.nf4_int4_gated_fwd(x, a, b, out_dtype=F32)
    assert_near(y, f * u, e * (1 + U24) + U24 * (f * u).abs() + 1e-38)
    assert torch.equal(y, nf4.nf4_int4_gated_fwd(x, a, b, out_dtype=F32))
