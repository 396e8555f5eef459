"""The products at the ends of the stated range of two scales' product: 2^-126
to 2^128, or 0. The bound is test_fp8_gpu's; codes from 1 up, so that no result
is subnormal."""
import pytest
import torch

import dequant_gemm_gb300 as nf4
from tests import test_fp8_gpu as products

pytestmark = pytest.mark.gpu
DEV, F8 = "cuda:0", torch.float8_e4m3fn


def codes(rows, cols, seed):
    """Codes of 1 to 448."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    return torch.randint(56, 127, (rows, cols), generator=g, dtype=torch.uint8).to(DEV).view(F8)


@pytest.mark.parametrize("M", [7, 40, 100, 300])
@pytest.mark.parametrize("dx", [False, True], ids=["fwd", "dx"])
@pytest.mark.parametrize("sa, sw", [(-100, -26), (-126, 0), (0, -126), (63, 37), (-40, 127), (127, -40)])
def test_products_at_the_ends_of_the_range(M, dx, sa, sw):
    """2^-126, and as large as the sums leave room for."""
    N, K = 144, 272
    red = N if dx else K
    a = nf4.FP8Tensor(codes(M, red, 1), torch.full((M, -(-red // 128)), 2.0 ** sa, device=DEV))
    w = nf4.FP8Tensor(codes(N, K, 2), torch.full((2, 3), -2.0 ** sw, device=DEV), 128)
    fn = nf4.nf4_fp8_matmul_bwd_dx if dx else nf4.nf4_fp8_matmul_fwd
    products.check_product(fn(a, w), a, w, dx, -(-red // 128))


@pytest.mark.parametrize("M", [7, 40, 100, 300])
def test_a_sum_of_zero_under_the_largest_factor(M):
    a = nf4.FP8Tensor(torch.zeros(M, 272, device=DEV).to(F8), torch.full((M, 3), 2.0 ** 64, device=DEV))
    w = nf4.FP8Tensor(codes(144, 272, 2), torch.full((2, 3), 2.0 ** 63, device=DEV), 128)
    assert not nf4.nf4_fp8_matmul_fwd(a, w).any()
