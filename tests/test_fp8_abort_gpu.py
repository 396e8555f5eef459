"""The 8-bit products' abort path where a CTA's copies are all under way before
the MMA issuer gives up: a CTA may only leave once they have landed in its
shared memory, also when the copying warp was done before the abort."""
import pytest
import torch

import dequant_gemm_gb300 as nf4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def quantized(rows, cols, seed, block_rows=1, std=1.0):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return nf4.nf4_fp8_quantize((torch.randn(rows, cols, generator=g) * std).to(DEV), block_rows=block_rows)


@pytest.mark.parametrize("dx", [False, True], ids=["fwd", "dx"])
@pytest.mark.parametrize("red", [128, 512])
@pytest.mark.parametrize("M", [8, 30, 60, 100, 700])
def test_abort_with_every_copy_under_way(M, red, dx):
    """A reduction no longer than the copy ring, a limit that the first copies
    outlast. What runs on the same SMs next comes out right, many times over."""
    cols = 2048
    w = quantized(red if dx else cols, cols if dx else red, 1, 128, 0.02)
    a = quantized(M, red, 2)
    fn = nf4.nf4_fp8_matmul_bwd_dx if dx else nf4.nf4_fp8_matmul_fwd
    want = fn(a, w)
    assert nf4.nf4_poll_device_status_site() == (0, 0)
    for _ in range(4):
        nf4.nf4_set_mma_wait_limit(200)
        try:
            fn(a, w)
            after = quantized(300, 512, 3)               # takes the SMs over at once
            status, site = nf4.nf4_poll_device_status_site()
        finally:
            nf4.nf4_set_mma_wait_limit(0)
        assert status == 7 and (site & 0xffffffff) >> 28 == (5 if dx else 4) and (site >> 24) & 15 == 2
        again = quantized(300, 512, 3)
        assert torch.equal(after.codes.view(torch.uint8), again.codes.view(torch.uint8))
        assert torch.equal(fn(a, w), want) and nf4.nf4_poll_device_status_site() == (0, 0)
