"""The 16-bit tensor-core kernels' abort path where a CTA's copies are all under
way before the MMA issuer gives up: a CTA may only leave once they have landed
in its shared memory, also when the copying warp was done before the abort."""
import pytest
import torch

import dequant_gemm_gb300 as nf4
from dequant_gemm_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dx", [False, True], ids=["fwd", "dx"])
@pytest.mark.parametrize("dtype", ["nf4", "int8"])
@pytest.mark.parametrize("red", [128, 384])
@pytest.mark.parametrize("M", [40, 100, 300])
def test_abort_with_every_copy_under_way(M, red, dtype, dx):
    """A reduction no longer than the copy ring (2 and 6 stages), a limit that
    the first copies outlast; the next calls on the same SMs come out right."""
    cols = 1024
    q = nf4.nf4_quantize(wl.weight(*((red, cols) if dx else (cols, red)), seed=1).to(DEV), dtype=dtype)
    x = wl.activations(M, red, seed=2).to(DEV)
    fn = nf4.nf4_matmul_bwd_dx if dx else nf4.nf4_matmul_fwd
    want = fn(x, q)
    assert nf4.nf4_poll_device_status_site() == (0, 0)
    for _ in range(4):
        nf4.nf4_set_mma_wait_limit(200)
        try:
            fn(x, q)
            status, site = nf4.nf4_poll_device_status_site()
        finally:
            nf4.nf4_set_mma_wait_limit(0)
        assert status == 7 and (site & 0xffffffff) >> 28 == (3 if dx else 2) and (site >> 24) & 15 == 2
        assert torch.equal(fn(x, q), want) and nf4.nf4_poll_device_status_site() == (0, 0)
