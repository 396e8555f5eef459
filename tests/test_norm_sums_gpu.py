"""Every element of a row enters the norm's sums once, at any length and in
every variant of the kernels.

Rows whose sum has one term that is not zero: adding zeros is exact, so the
bounds do not grow with the length, and a sum that misses an element, or takes
one twice, is off by all of it. u = 2^-24.
  Forward, h = v at one column: v^2, the division by the length and the addition
  of eps round once each, which the root halves; the reciprocal root is within
  2 ulp (4 u): 6 u for rstd. y takes two products more, then its type's rounding.
  Backward, dy = g at one column j of a dense row: mean(g xh) rounds four times,
  dx_k = -rstd xh_k mean four times more: 10 u; the term rstd g w of column j is
  within 4 u. dweight: products of three factors (2 u) and one rounding for each
  addition of a term that is not zero."""
import pytest
import torch

import dequant_gemm_gb300 as nf4
from tests import test_norm_gpu as dense

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF_ULP, TINY, U, EPS = dense.HALF_ULP, dense.TINY, 2.0 ** -24, 1e-6


def columns(cols, seed):
    """All columns of a short row; of a long one its ends, the surroundings of
    multiples of 1024 and 700 others; in random order, so that the rows that
    have them lie at every offset."""
    g = torch.Generator().manual_seed(seed)
    c = torch.arange(cols)
    if cols > 1200:
        near = (c % 1024 < 9) | (c % 1024 >= 1015)
        ends = (c < 40) | (c >= cols - 40)
        some = torch.zeros(cols, dtype=torch.bool)
        some[torch.randperm(cols, generator=g)[:700]] = True
        c = c[ends | some | (near & (torch.rand(cols, generator=g) < 1200 / (cols / 57 + 1200)))]
    return c[torch.randperm(len(c), generator=g)].to(DEV)


def normal(*shape, seed, dtype=F32):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(dtype)


# the forms in registers and the two-pass ones, even and odd, and the borders between them
LENGTHS = [1, 7, 24, 257, 528, 1023, 2047, 2048, 3584, 4097, 5001, 5119, 5376, 5384, 6000, 8177, 8179,
           8184, 8192, 8200, 12000, 16377, 16379, 16384, 16392, 20000, 32768, 32776, 70001]


@pytest.mark.parametrize("cols", LENGTHS)
@pytest.mark.parametrize("dtype, res_dtype", [(F32, None), (BF16, F32), (F16, F16), (BF16, None)])
def test_forward_takes_every_element_once(cols, dtype, res_dtype):
    w = normal(cols, seed=1).abs() + 0.5
    for seed in (2, 3):
        hot = columns(cols, seed)
        rows = len(hot)
        at = (torch.arange(rows, device=DEV), hot)
        x = torch.zeros(rows, cols, dtype=dtype, device=DEV)
        x[at] = (normal(rows, seed=seed + 4).abs() * 30 + 1).to(dtype)
        res = None if res_dtype is None else torch.zeros(rows, cols, dtype=res_dtype, device=DEV)
        if res is not None:
            res[at] = normal(rows, seed=seed + 6).abs().to(res_dtype)
        y, h, rstd = nf4.nf4_rmsnorm_fwd(x, w, res, eps=EPS, save_rstd=True)
        v = x[at] if res is None else (x[at].float() + res[at].float()).to(res_dtype)
        assert torch.equal(h[at], v)
        ref = 1 / torch.sqrt(v.double() ** 2 / cols + EPS)
        assert ((rstd.double() - ref).abs() <= 6 * U * ref).all()
        ref = v.double() * ref * w[hot].double()
        assert ((y[at].double() - ref).abs() <= (8 * U + HALF_ULP[dtype] * (1 + 8 * U)) * ref + TINY[dtype]).all()
        y[at] = 0
        assert not y.any()


@pytest.mark.parametrize("cols", LENGTHS)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_backward_takes_every_element_once(cols, dtype):
    """One column of dy a row. Then few columns that many rows share, so that
    dweight adds up the rows of each CTA and the CTAs."""
    w = 1 + 0.1 * normal(cols, seed=1)
    for shared in (False, True):
        hot = columns(cols, 5)
        if shared:
            hot = hot[:5].repeat(-(-500 // min(5, len(hot))))[:500]
        rows = len(hot)
        at = (torch.arange(rows, device=DEV), hot)
        h = normal(rows, cols, seed=2, dtype=dtype)
        rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
        dy = torch.zeros(rows, cols, dtype=dtype, device=DEV)
        dy[at] = (normal(rows, seed=3).sign() * (1 + normal(rows, seed=4).abs().clamp(max=2)) * min(cols, 8192)).to(dtype)
        dx, dw = nf4.nf4_rmsnorm_bwd(dy, h, w, rstd)
        R, G, W = rstd.double(), dy[at].double(), w.double()
        terms = G * h[at].double() * R                               # of dweight
        mean = terms * W[hot] / cols
        for lo in range(0, rows, 400):                               # (64-bit copies of a part at a time)
            s = slice(lo, min(lo + 400, rows))
            ref = -R[s, None] * (h[s].double() * R[s, None]) * mean[s, None]
            bound = 10 * U * ref.abs()
            here = (torch.arange(ref.shape[0], device=DEV), hot[s])
            ref[here] += R[s] * G[s] * W[hot[s]]
            bound[here] += 4 * U * (R[s] * G[s] * W[hot[s]]).abs()
            bound = bound * (1 + HALF_ULP[dtype]) + HALF_ULP[dtype] * ref.abs() + TINY[dtype]
            assert ((dx[s].double() - ref).abs() <= bound).all()
        zero = torch.zeros(cols, dtype=torch.float64, device=DEV)
        ref, size = zero.index_add(0, hot, terms), zero.index_add(0, hot, terms.abs())
        count = zero.index_add(0, hot, torch.ones_like(terms))
        assert ((dw.double() - ref).abs() <= (count + 3) * U * size).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows, cols", [(400, 5384), (400, 8192), (400, 8200), (330, 12000), (330, 16384), (320, 16392),
                                        (330, 9001), (310, 20001)])
def test_backward_of_long_rows_with_more_rows_than_ctas(rows, cols, dtype):
    """Dense rows: the forms for long rows with several rows a CTA."""
    dense.test_backward(rows, cols, dtype, True)
