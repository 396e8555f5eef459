"""What the norm's Python calls refuse on GPU tensors: an operand off a 16-byte
boundary, by its name. (The refusals that need no device are tested on the CPU.)"""
import pytest
import torch

import dequant_gemm_gb300 as nf4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_operands_off_the_16_byte_grid_are_named():
    good = {n: torch.ones(4, 41, device=DEV) for n in ("x", "residual", "out_h", "dy", "h", "dh")}
    good["weight"] = torch.ones(41, device=DEV)
    off = {n: torch.ones(5, 41, device=DEV)[1:] for n in good}
    off["weight"] = torch.ones(42, device=DEV)[1:]
    rstd = torch.ones(5, device=DEV)[1:]           # fp32 values need no more than their own alignment

    def fwd(x, weight, residual, out_h):
        return nf4.nf4_rmsnorm_fwd(x, weight, residual, out_h=out_h)

    def bwd(dy, h, weight, dh):
        return nf4.nf4_rmsnorm_bwd(dy, h, weight, rstd, dh=dh)

    for call, names in ((fwd, ("x", "weight", "residual", "out_h")), (bwd, ("dy", "h", "weight", "dh"))):
        call(**{n: good[n] for n in names})
        for bad in names:
            with pytest.raises(ValueError, match=f"^{bad} must start on a 16-byte boundary"):
                call(**{n: (off if n == bad else good)[n] for n in names})
