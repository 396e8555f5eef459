"""The RMS norm on the GPU against the 64-bit oracle.

Bounds, per element, u = 2^-24: the fp32 mean of n squares is off by at most
(n + 2) u relative in any order of summation, rstd by half of that and 4 u for
its own rounding, y by 2 u more; then half an ulp of y's type. Gradients are
sums of exactly known terms: (n + 16) u of the sum of their magnitudes."""
import numpy as np
import pytest
import torch

import dequant_gemm_gb300 as nf4
from oracle import fp8_oracle as o

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8, F32, BF16, F16 = torch.float8_e4m3fn, torch.float32, torch.bfloat16, torch.float16
HALF_ULP = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {F32: 2.0 ** -149, BF16: 2.0 ** -133, F16: 2.0 ** -24}
EPS = 1e-6


def make(rows, cols, seed, dtype=F32, std=1.0):
    g = torch.Generator(device="cpu").manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * std
    x[:, cols // 3] *= 20
    return x.to(dtype)


def y_bound(ref, cols, dtype):
    rel = ((cols + 2) / 2 + 6) * 2.0 ** -24
    return np.abs(ref) * (rel + HALF_ULP[dtype] * (1 + rel)) + TINY[dtype]


TYPES = [(F32, None), (F32, F32), (BF16, None), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)]


@pytest.mark.parametrize("x_dtype, res_dtype", TYPES)
@pytest.mark.parametrize("rows, cols", [(1, 1), (3, 7), (2, 24), (5, 257), (1, 3584), (700, 512),
                                        (9, 1040), (3, 5001), (2, 8192), (2, 20000), (1, 70001)])
def test_forward(rows, cols, x_dtype, res_dtype):
    x, w = make(rows, cols, cols, x_dtype), 1 + make(1, cols, 2, std=0.1)[0]
    res = None if res_dtype is None else make(rows, cols, 3, res_dtype)
    h_ref = x if res is None else (x.float() + res.float()).to(res_dtype)
    for out in (x_dtype, F32, BF16):
        y, h, rstd = nf4.nf4_rmsnorm_fwd(x.to(DEV), w.to(x_dtype).to(DEV), None if res is None else res.to(DEV),
                                         eps=EPS, out_dtype=out, save_rstd=True)
        assert torch.equal(h.cpu(), h_ref) and y.dtype == out
        ref, r_ref = o.rmsnorm(h_ref.double().numpy(), w.to(x_dtype).double().numpy(), EPS)
        assert (np.abs(y.double().cpu().numpy() - ref) <= y_bound(ref, cols, out)).all()
        assert (np.abs(rstd.double().cpu().numpy() - r_ref) <= r_ref * ((cols + 2) / 2 + 4) * 2.0 ** -24).all()


@pytest.mark.parametrize("rows, cols", [(1, 16), (1, 3584), (6, 144), (300, 1040), (2, 16384), (2, 40000)])
@pytest.mark.parametrize("x_dtype, res_dtype", [(BF16, BF16), (BF16, F32), (F32, None)])
def test_8bit_output_is_the_32bit_output_quantized(rows, cols, x_dtype, res_dtype):
    """The fused codes and scales equal quantizing the kernel's own fp32 output,
    which test_forward holds to the oracle; a zero row gives zeros."""
    x, w = make(rows, cols, cols, x_dtype).to(DEV), (1 + make(1, cols, 2, std=0.1)[0]).to(DEV)
    res = None if res_dtype is None else make(rows, cols, 3, res_dtype).to(DEV)
    if rows > 1:
        x[-1] = 0
        if res is not None:
            res[-1] = 0
    q, h, _ = nf4.nf4_rmsnorm_fwd(x, w, res, eps=EPS, out_dtype=F8)
    y, h2, _ = nf4.nf4_rmsnorm_fwd(x, w, res, eps=EPS, out_dtype=F32)
    codes, scale = o.quantize(y.cpu().numpy(), 1)
    assert np.array_equal(q.codes.view(torch.uint8).cpu().numpy(), codes)
    assert np.array_equal(q.scale.cpu().numpy(), scale) and torch.equal(h, h2)
    if rows > 1:
        assert not q.scale[-1].any() and not (codes[-1] & 127).any()   # (a negative weight gives -0)


def test_stream_updated_in_place():
    x, res, w = make(40, 528, 1, BF16).to(DEV), make(40, 528, 2).to(DEV), torch.ones(528, device=DEV)
    y, h, _ = nf4.nf4_rmsnorm_fwd(x, w, res.clone(), out_dtype=F8)
    y2, h2, _ = nf4.nf4_rmsnorm_fwd(x, w, res, out_dtype=F8, out_h=res)
    assert h2 is res and torch.equal(h, res) and torch.equal(y.scale, y2.scale)
    assert torch.equal(y.codes.view(torch.uint8), y2.codes.view(torch.uint8))


def test_nan_and_infinite_rows_stay_in_their_rows():
    x, w = make(6, 272, 1).to(DEV), torch.ones(272, device=DEV)
    x[1, 5], x[2, 200] = float("nan"), float("inf")
    for out in (F32, F8):
        y, _, _ = nf4.nf4_rmsnorm_fwd(x, w, out_dtype=out)
        v = y if out == F32 else nf4.nf4_fp8_dequantize(y)
        assert v[1].isnan().all() and v[2, 200].isnan()
        assert not v[0].isnan().any() and not v[3:].isnan().any()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows, cols", [(1, 1), (1, 3584), (3, 7), (5, 257), (700, 512), (333, 5001),
                                        (1200, 528), (9, 16384), (2, 40000), (2, 70001)])
@pytest.mark.parametrize("with_dh", [False, True])
def test_backward(rows, cols, dtype, with_dh):
    h, dy = make(rows, cols, 1, dtype), make(rows, cols, 2, dtype, std=0.1)
    dh = make(rows, cols, 3, dtype, std=0.1) if with_dh else None
    for w_dtype in {F32, dtype}:
        w = (1 + make(1, cols, 4, std=0.1)[0]).to(w_dtype)
        H, G, W = h.double().numpy(), dy.double().numpy(), w.double().numpy()
        rstd = torch.from_numpy(o.rmsnorm(H, W, EPS)[1]).float()
        R = rstd.double().numpy()[:, None]
        dx, dw = nf4.nf4_rmsnorm_bwd(dy.to(DEV), h.to(DEV), w.to(DEV), rstd.to(DEV),
                                     dh=None if dh is None else dh.to(DEV))
        ref, w_ref = o.rmsnorm_grads(G, H, W, EPS, None if dh is None else dh.double().numpy())
        xh = H * R
        terms = R * (np.abs(G * W) + np.abs(xh) * np.abs(G * W * xh).mean(axis=1, keepdims=True))
        bound = (cols + 16) * 2.0 ** -24 * terms
        if dh is not None:
            bound = bound + 2 * 2.0 ** -24 * np.abs(dh.double().numpy())
        bound = bound * (1 + HALF_ULP[dtype]) + HALF_ULP[dtype] * np.abs(ref) + TINY[dtype]
        assert dx.dtype == dtype and dw.dtype == w_dtype
        assert (np.abs(dx.double().cpu().numpy() - ref) <= bound).all()
        bound = (rows + 16) * 2.0 ** -24 * np.abs(G * xh).sum(axis=0)
        bound = bound * (1 + HALF_ULP[w_dtype]) + HALF_ULP[w_dtype] * np.abs(w_ref) + TINY[w_dtype]
        assert (np.abs(dw.double().cpu().numpy() - w_ref) <= bound).all()
        again = nf4.nf4_rmsnorm_bwd(dy.to(DEV), h.to(DEV), w.to(DEV), rstd.to(DEV),
                                    dh=None if dh is None else dh.to(DEV))
        assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


def test_backward_against_differences():
    """The kernel's gradients against central differences of the 64-bit forward
    (error of the differences below 1e-6, of the fp32 kernel below 1e-4 of the
    terms' size at these sizes)."""
    rows, cols = 5, 96
    h, dy, w = make(rows, cols, 1), make(rows, cols, 2), 1 + make(1, cols, 4, std=0.1)[0]
    H, G, W = (t.double().numpy() for t in (h, dy, w))
    rstd = torch.from_numpy(o.rmsnorm(H, W, EPS)[1]).float()
    dx, dw = (t.double().cpu().numpy() for t in nf4.nf4_rmsnorm_bwd(dy.to(DEV), h.to(DEV), w.to(DEV),
                                                                   rstd.to(DEV)))
    g, step = np.random.default_rng(0), 1e-5
    for _ in range(6):
        v, u = g.normal(size=H.shape), g.normal(size=W.shape)
        loss = lambda a, b: (G * o.rmsnorm(a, b, EPS)[0]).sum()  # noqa: E731
        num = (loss(H + step * v, W) - loss(H - step * v, W)) / (2 * step)
        assert abs(num - (dx * v).sum()) <= 1e-4 * np.abs(dx * v).sum()
        num = (loss(H, W + step * u) - loss(H, W - step * u)) / (2 * step)
        assert abs(num - (dw * u).sum()) <= 1e-4 * np.abs(dw * u).sum()


def test_empty_batches():
    x, w = torch.empty(0, 64, device=DEV), torch.ones(64, device=DEV)
    y, h, rstd = nf4.nf4_rmsnorm_fwd(x, w, x, out_dtype=F8, save_rstd=True)
    assert y.rows == 0 and h.shape == (0, 64) and rstd.shape == (0,)
    dx, dw = nf4.nf4_rmsnorm_bwd(x, x, w, torch.empty(0, device=DEV))
    assert dx.shape == (0, 64) and (dw == 0).all()


def test_offsets_beyond_32_bits():
    rows, cols = 600_000, 4096
    x = torch.zeros(rows, cols, dtype=BF16, device=DEV)
    x[-8:] = make(8, cols, 1, BF16).to(DEV)
    w = torch.ones(cols, device=DEV)
    y, _, rstd = nf4.nf4_rmsnorm_fwd(x, w, out_dtype=F8, save_rstd=True)
    tail, _, r = nf4.nf4_rmsnorm_fwd(x[-8:].contiguous(), w, out_dtype=F8, save_rstd=True)
    assert torch.equal(y.codes[-8:].view(torch.uint8), tail.codes.view(torch.uint8))
    assert torch.equal(y.scale[-8:], tail.scale) and torch.equal(rstd[-8:], r)
    assert not y.scale[:-8].any()
    dy = torch.zeros_like(x)
    dy[-8:] = make(8, cols, 2, BF16).to(DEV)
    dx, dw = nf4.nf4_rmsnorm_bwd(dy, x, w, rstd)
    dx8, dw8 = nf4.nf4_rmsnorm_bwd(dy[-8:].contiguous(), x[-8:].contiguous(), w, r)
    assert torch.equal(dx[-8:], dx8) and not dx[:-8].any()
    assert ((dw - dw8).abs() <= 24 * 2.0 ** -24 * (dy[-8:].float() * x[-8:].float() * r[:, None]).abs().sum(0)).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows, cols", [(5, 2047), (4, 4097), (3, 8185), (3, 8187), (3, 16377), (2, 16379)])
def test_forward_at_the_borders_of_odd_lengths(rows, cols, dtype):
    """One and two runs a thread, and rows read twice: 1024 and 2048 runs."""
    test_forward(rows, cols, dtype, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows, cols", [(1300, 129), (1000, 1023), (1250, 1024), (500, 2047), (310, 5119),
                                        (160, 5363), (160, 5371), (9, 8185), (9, 8187)])
def test_backward_with_more_rows_than_ctas(rows, cols, dtype):
    """Rows beyond the CTAs that run at once, at lengths next to where their
    number or the threads' runs change."""
    test_backward(rows, cols, dtype, True)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("cols", [13, 1023, 5119, 8187])
def test_rows_do_not_see_their_neighbours(cols, dtype):
    """An odd length's 16-byte accesses reach into the rows beside it: what is
    there, finite or NaN, changes no bit of a row in its place (on which, modulo
    8 rows, the order of an odd row's sums depends)."""
    rows = 17
    x, w = make(1, cols, 1, dtype).to(DEV), (1 + make(1, cols, 2, std=0.1)[0]).to(DEV)
    res, dy, dh = (make(1, cols, s, dtype).to(DEV) for s in (3, 4, 5))

    def run(neighbours):
        def among(row):
            full = torch.full((rows, cols), neighbours, dtype=row.dtype, device=DEV)
            full[1::2] = row
            return full

        y, h, r = nf4.nf4_rmsnorm_fwd(among(x), w, among(res), save_rstd=True)
        dx, dw = nf4.nf4_rmsnorm_bwd(among(dy), h, w, r, dh=among(dh))
        return (y, h, r, dx), dw

    (clean, _), (nans, dw) = run(3.0), run(float("nan"))
    for many, one in zip(nans, clean):
        assert many[0::2].isnan().all() and not one.isnan().any()
        assert torch.equal(many[1::2], one[1::2])
    assert dw.isnan().all()
