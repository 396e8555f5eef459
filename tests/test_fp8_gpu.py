"""The 8-bit quantizer and products on the GPU against the oracle.

Quantized codes and scales have to match bit for bit. A product's error bound
is derived per element: the 128 products of a block are exact in fp32 and are
summed with at most one fp32 rounding or truncation (2^-23) each, the two
scales, their product with the sum and the addition to the total round once
each (2^-24), so |Y - Y_ref| <= (128 * 2^-23 + (3 + blocks) * 2^-24) * sum of
|products|, plus half an ulp (2^-8 relative) where Y is bf16 and 2^-24 |Y|
each for adding to an output."""
import numpy as np
import pytest
import torch

import dequant_gemm_gb300 as nf4
from oracle import fp8_oracle as o

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn


def make(rows, cols, seed, std=1.0, dtype=torch.float32):
    g = torch.Generator(device="cpu").manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * std
    x[:, torch.randint(0, cols, (max(1, cols // 200),), generator=g)] *= 20
    return x.to(dtype)


def codes_of(q):
    return q.codes.view(torch.uint8).cpu().numpy()


def assert_same(q, codes, scale):
    assert np.array_equal(q.scale.cpu().numpy(), scale, equal_nan=True)
    got = codes_of(q)
    nan = (codes & 127) == 127
    assert np.array_equal(got[~nan], codes[~nan]) and ((got[nan] & 127) == 127).all()


def values64(q):
    """fp64 values on the GPU, from the oracle's code table."""
    table = torch.from_numpy(o.VALUES).to(DEV)
    s = q.scale.double().repeat_interleave(q.block_rows, 0)[:q.rows]
    return table[q.codes.view(torch.uint8).long()] * s.repeat_interleave(128, 1)[:, :q.cols]


def check_product(got, a, w, dx, blocks, before=None):
    A, W = values64(a), values64(w)
    W = W if dx else W.t()
    ref, terms = A @ W, A.abs() @ W.abs()
    bound = (128 * 2.0 ** -23 + (3 + blocks) * 2.0 ** -24) * terms
    if before is not None:
        ref = ref + before.double()
        bound = bound + 2.0 ** -24 * (ref.abs() + before.double().abs())
    if got.dtype == torch.bfloat16:
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
    bad = (got.double() - ref).abs() > bound
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, first {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows, cols", [(1, 16), (1, 128), (3, 144), (130, 256), (257, 1040)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_is_bit_exact(rows, cols, block_rows, dtype):
    x = make(rows, cols, rows + cols, dtype=dtype)
    x[rows // 2] = 0
    q = nf4.nf4_fp8_quantize(x.to(DEV), block_rows=block_rows)
    assert_same(q, *o.quantize(x.float().numpy(), block_rows))
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        v = nf4.nf4_fp8_dequantize(q, out_dtype=dt)
        s = q.scale.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
        assert torch.equal(v, (q.codes.float() * s).to(dt))


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_of_extreme_values(block_rows):
    x = torch.zeros(260, 400)
    x[0, 0], x[0, 130], x[0, 260] = 3.3e38, 2.0 ** -117, 2.0 ** -118
    x[130, 1], x[130, 129], x[131, 129] = float("inf"), float("nan"), 1.0
    x[259, 399], x[259, 398] = -1e-30, 3e-33
    q = nf4.nf4_fp8_quantize(x.to(DEV), block_rows=block_rows)
    assert_same(q, *o.quantize(x.numpy(), block_rows))
    v = nf4.nf4_fp8_dequantize(q)
    assert v[130, :128].isnan().all() and v[130, 128:256].isnan().all() and not v[130, 256:].isnan().any()
    assert v[129].isnan().any() == (block_rows == 128) and not v[:128].isnan().any()


SHAPES = [(1, 16, 16), (300, 16, 16), (1, 512, 4096), (2, 144, 272), (5, 4096, 528), (16, 272, 1040), (17, 256, 128),
          (33, 1040, 400), (64, 528, 2064), (65, 128, 144), (100, 2048, 640), (128, 272, 272),
          (129, 400, 528), (250, 512, 896), (300, 1040, 1552), (513, 2064, 1040), (1000, 784, 3600)]


@pytest.mark.parametrize("M, N, K", SHAPES)
@pytest.mark.parametrize("dx", [False, True], ids=["fwd", "dx"])
def test_product(M, N, K, dx):
    red = N if dx else K
    a = nf4.nf4_fp8_quantize(make(M, red, M + N, dtype=torch.bfloat16).to(DEV))
    w = nf4.nf4_fp8_quantize(make(N, K, N + K, std=0.02).to(DEV), block_rows=128)
    fn = nf4.nf4_fp8_matmul_bwd_dx if dx else nf4.nf4_fp8_matmul_fwd
    blocks = -(-red // 128)
    for dt in (torch.float32, torch.bfloat16):
        y = fn(a, w, out_dtype=dt)
        check_product(y, a, w, dx, blocks)
        assert torch.equal(y, fn(a, w, out_dtype=dt))              # repeatable
        out = make(M, K if dx else N, 9).to(dt).to(DEV)
        before = out.clone()
        assert fn(a, w, out=out, accumulate=True) is out
        check_product(out, a, w, dx, blocks, before)
    assert nf4.nf4_poll_device_status() == 0


@pytest.mark.parametrize("M", [3, 40, 300])
@pytest.mark.parametrize("dx", [False, True], ids=["fwd", "dx"])
def test_one_hot_rows_return_the_weight(M, dx):
    """One code of 1.0 a row: Y is one weight value, exact up to the scales'
    two roundings; every weight row (column) is hit where M allows."""
    N, K = 272, 400
    red = N if dx else K
    w = nf4.nf4_fp8_quantize(make(N, K, 5, std=0.02).to(DEV), block_rows=128)
    codes = torch.zeros(M, red, device=DEV)
    at = (torch.arange(M, device=DEV) * 7) % red
    codes[torch.arange(M, device=DEV), at] = 1.0
    scale = torch.rand(M, -(-red // 128), device=DEV) + 0.5
    a = nf4.FP8Tensor(codes.to(F8), scale)
    y = (nf4.nf4_fp8_matmul_bwd_dx if dx else nf4.nf4_fp8_matmul_fwd)(a, w)
    W = values64(w) if dx else values64(w).t()
    ref = W[at] * scale.double()[torch.arange(M, device=DEV), at // 128][:, None]
    assert ((y.double() - ref).abs() <= 3 * 2.0 ** -24 * ref.abs()).all()


@pytest.mark.parametrize("M", [4, 50, 290])
def test_nan_and_zero_rows_stay_in_their_rows(M):
    w = nf4.nf4_fp8_quantize(make(272, 400, 5, std=0.02).to(DEV), block_rows=128)
    x = make(M, 400, 6)
    x[1, 300], x[2] = float("nan"), 0.0
    y = nf4.nf4_fp8_matmul_fwd(nf4.nf4_fp8_quantize(x.to(DEV)), w)
    assert y[1].isnan().all() and (y[2] == 0).all()
    assert not y[0].isnan().any() and not y[3:].isnan().any()


def test_scales_of_any_size_multiply_as_they_are():
    """Hand-made scales (zero, negative, large) and codes at the type's ends."""
    g = torch.Generator(device="cpu").manual_seed(3)
    for M in (7, 40, 200):
        a = nf4.FP8Tensor(torch.randint(0, 127, (M, 272), generator=g, dtype=torch.uint8).to(DEV).view(F8),
                          (torch.randn(M, 3, generator=g) * 1e10).to(DEV))
        w = nf4.FP8Tensor(torch.randint(0, 127, (144, 272), generator=g, dtype=torch.uint8).to(DEV).view(F8),
                          torch.tensor([[0.0, -1e-10, 1e4], [1.0, 2.0 ** -120, 0.0]], device=DEV), 128)
        check_product(nf4.nf4_fp8_matmul_fwd(a, w), a, w, False, 3)


@pytest.mark.parametrize("M", [7, 40, 100, 300])
def test_scales_whose_product_alone_is_in_range(M):
    """Neither scale times a block's sum fits fp32; the two scales' product does."""
    for sa, sw in ((1e-34, 1e34), (1e34, 1e-34)):
        a = nf4.FP8Tensor(torch.full((M, 272), 448.0, device=DEV).to(F8), torch.full((M, 3), sa, device=DEV))
        w = nf4.FP8Tensor(torch.full((144, 272), 448.0, device=DEV).to(F8),
                          torch.full((2, 3), sw, device=DEV), 128)
        check_product(nf4.nf4_fp8_matmul_fwd(a, w), a, w, False, 3)


def test_empty_calls():
    w = nf4.nf4_fp8_quantize(make(32, 256, 5).to(DEV), block_rows=128)
    assert nf4.nf4_fp8_matmul_fwd(nf4.alloc_fp8(0, 256, DEV), w).shape == (0, 32)
    none = nf4.alloc_fp8(0, 256, DEV, 128)
    assert nf4.nf4_fp8_matmul_fwd(nf4.alloc_fp8(3, 256, DEV), none).shape == (3, 0)
    dy = nf4.alloc_fp8(3, 0, DEV)
    assert (nf4.nf4_fp8_matmul_bwd_dx(dy, none) == 0).all()       # an empty reduction
    assert nf4.nf4_fp8_quantize(torch.empty(0, 32, device=DEV)).rows == 0
    assert nf4.nf4_fp8_dequantize(nf4.alloc_fp8(0, 32, DEV)).shape == (0, 32)


def test_row_slices_and_another_stream():
    """Rows of a larger activation (codes and scales sliced), on a side stream."""
    w = nf4.nf4_fp8_quantize(make(256, 400, 5, std=0.02).to(DEV), block_rows=128)
    q = nf4.nf4_fp8_quantize(make(50, 400, 6).to(DEV))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for lo, hi in ((1, 2), (7, 50), (3, 20)):
            part = nf4.FP8Tensor(q.codes[lo:hi], q.scale[lo:hi])
            check_product(nf4.nf4_fp8_matmul_fwd(part, w), part, w, False, 4)
    side.synchronize()


def test_offsets_beyond_32_bits():
    """Codes and outputs of more than 2^31 elements: the last rows come out right."""
    rows, cols = 140_000, 16_384
    q = nf4.alloc_fp8(rows, cols, DEV)
    x = make(64, cols, 8, dtype=torch.bfloat16).to(DEV)
    big = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    big[-64:] = x
    nf4.nf4_fp8_quantize(big, out=q)
    tail = nf4.nf4_fp8_quantize(x)
    assert torch.equal(q.codes[-64:].view(torch.uint8), tail.codes.view(torch.uint8))
    assert torch.equal(q.scale[-64:], tail.scale) and not q.scale[:-64].any()
    del big
    w = nf4.nf4_fp8_quantize(make(32, cols, 9, std=0.02).to(DEV), block_rows=128)
    y = nf4.nf4_fp8_matmul_fwd(q, w, out_dtype=torch.bfloat16)
    check_product(y[-64:], tail, w, False, 128)
    assert not y[:-64].any()
    dy = nf4.nf4_fp8_quantize(make(64, 32, 10).to(DEV))
    all_dy = nf4.alloc_fp8(rows, 32, DEV)
    all_dy.codes.view(torch.uint8).zero_()
    all_dy.scale.fill_(1.0)
    all_dy.codes[-64:], all_dy.scale[-64:] = dy.codes, dy.scale
    dx = nf4.nf4_fp8_matmul_bwd_dx(all_dy, w, out_dtype=torch.bfloat16)
    check_product(dx[-64:], dy, w, True, 1)
    assert not dx[:-64].any()


def test_gradient_is_the_forwards_adjoint():
    """<dY, Y(X)> = <dX, X> for the linear map X -> Y, both from the kernels:
    each side is off by at most its products' bounds."""
    M, N, K = 96, 528, 400
    x = nf4.nf4_fp8_quantize(make(M, K, 1).to(DEV))
    dy = nf4.nf4_fp8_quantize(make(M, N, 2).to(DEV))
    w = nf4.nf4_fp8_quantize(make(N, K, 3, std=0.02).to(DEV), block_rows=128)
    X, G, W = values64(x), values64(dy), values64(w)
    left = (G * nf4.nf4_fp8_matmul_fwd(x, w).double()).sum()
    right = (X * nf4.nf4_fp8_matmul_bwd_dx(dy, w).double()).sum()
    terms = (G.abs() * (X.abs() @ W.abs().t())).sum()
    assert abs(left - right) <= 2 * (128 * 2.0 ** -23 + 8 * 2.0 ** -24) * terms
