"""Refusals of the 8-bit operators and the RMS norm: the Python checks on CPU
tensors, and the C entry points' host-side validation (no device touched)."""
import ctypes

import pytest
import torch

import dequant_gemm_gb300 as nf4

P = 1 << 20   # a fake aligned address, never dereferenced by validation
FP8 = torch.float8_e4m3fn


def act(rows=4, cols=256):
    return nf4.alloc_fp8(rows, cols, "cpu")


def weight(rows=32, cols=256):
    return nf4.alloc_fp8(rows, cols, "cpu", block_rows=128)


@pytest.mark.parametrize("kw, match", [
    (dict(x=torch.zeros(4, 32, dtype=torch.int8)), "float32"),
    (dict(x=torch.zeros(4, 24)), "multiple of 16"),
    (dict(x=torch.zeros(2, 4, 32)), "2-D"),
    (dict(x=torch.zeros(32, 4).t()), "contiguous"),
    (dict(x=torch.zeros(4, 32), block_rows=64), "block_rows"),
    (dict(x=torch.zeros(4, 256), out=nf4.alloc_fp8(4, 128, "cpu")), "asked for"),
    (dict(x=torch.zeros(4, 256), out=nf4.alloc_fp8(4, 256, "cpu", 128)), "asked for"),
    (dict(x=torch.zeros(4, 32)), "CUDA device"),
])
def test_quantize_refuses(kw, match):
    with pytest.raises(ValueError, match=match):
        nf4.nf4_fp8_quantize(**kw)


def test_matmul_refuses():
    fwd, dx = nf4.nf4_fp8_matmul_fwd, nf4.nf4_fp8_matmul_bwd_dx
    a, w = act(), weight()
    for bad, match in ((torch.zeros(4, 256), "FP8Tensor"), (act(cols=128), "must be"),
                       (nf4.FP8Tensor(a.codes.view(torch.uint8), a.scale), "float8"),
                       (nf4.FP8Tensor(a.codes, a.scale[:, :1].contiguous()), "shape"),
                       (nf4.FP8Tensor(a.codes, a.scale.double()), "float32"),
                       (nf4.alloc_fp8(4, 256, "cpu", 128), "block_rows")):
        with pytest.raises(ValueError, match=match):
            fwd(bad, w)
    with pytest.raises(ValueError, match="block_rows"):
        fwd(a, act(32))
    with pytest.raises(ValueError, match="multiple of 16"):
        fwd(a, weight(rows=24))
    with pytest.raises(ValueError, match="must be"):
        dx(a, w)                                   # dY must be [M, rows]
    with pytest.raises(ValueError, match="shape"):
        fwd(a, w, out=torch.empty(4, 31))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        fwd(a, w, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="accumulate"):
        dx(act(cols=32), w, accumulate=True)
    with pytest.raises(ValueError, match="expected cpu"):
        fwd(a, nf4.alloc_fp8(32, 256, "meta", 128))
    with pytest.raises(ValueError, match="CUDA device"):
        fwd(a, w)


def test_norm_refuses():
    x, w = torch.zeros(4, 32, dtype=torch.bfloat16), torch.ones(32)
    f = nf4.nf4_rmsnorm_fwd
    for args, kw, match in (((x.int(), w), {}, "float32"), ((x, w[:16]), {}, "shape"),
                            ((x.t(), w[:4]), {}, "contiguous"),
                            ((x[:, :0].contiguous(), w[:0]), {}, "cols > 0"),
                            ((x, w, x.half()), {}, "residual"), ((x, w, x[:2]), {}, "shape"),
                            ((x, w), dict(out_h=x), "out_h"), ((x, w), dict(eps=-1.0), "eps"),
                            ((x, w), dict(eps=float("nan")), "eps"),
                            ((x, w), dict(out_dtype=torch.int8), "output"),
                            ((x, w, x), dict(out_h=torch.zeros(4, 32)), "out_h"),
                            ((x[:, :24].contiguous(), w[:24]), dict(out_dtype=FP8), "multiple of 16"),
                            ((x, w), {}, "CUDA device")):
        with pytest.raises(ValueError, match=match):
            f(*args, **kw)
    b, r = nf4.nf4_rmsnorm_bwd, torch.ones(4)
    for args, kw, match in (((x.float(), x, w, r), {}, "dy"), ((x, x, w, r[:3]), {}, "rstd"),
                            ((x, x, w, r), dict(dh=x.float()), "dh"), ((x, x, w, r), {}, "CUDA device")):
        with pytest.raises(ValueError, match=match):
            b(*args, **kw)


def _t(codes=P, scale=P, rows=32, cols=256, block_rows=128):
    return nf4.nf4_fp8_tensor(codes, scale, rows, cols, block_rows)


def test_c_abi_validates_products():
    L = nf4.lib()
    f, d = L.nf4_fp8_matmul_fwd, L.nf4_fp8_matmul_bwd_dx
    a, w = ctypes.byref(_t(rows=4, block_rows=1)), ctypes.byref(_t())
    assert f(None, w, P, 0, 0, None) == 1 and f(a, None, P, 0, 0, None) == 1
    assert f(a, w, None, 0, 0, None) == 1
    assert f(w, w, P, 0, 0, None) == 4 and f(a, a, P, 0, 0, None) == 4
    assert f(a, w, P, 2, 0, None) == 2 and f(a, w, P, 0, 2, None) == 2     # element type, flags
    assert f(a, ctypes.byref(_t(rows=24)), P, 0, 0, None) == 2
    assert f(ctypes.byref(_t(rows=4, cols=128, block_rows=1)), w, P, 0, 0, None) == 2
    assert f(ctypes.byref(_t(rows=-1, block_rows=1)), w, P, 0, 0, None) == 2
    assert d(a, w, P, 0, 0, None) == 2
    assert f(ctypes.byref(_t(rows=1 << 31, block_rows=1)), w, P, 0, 0, None) == 2
    assert f(a, w, P + 4, 0, 0, None) == 3
    assert f(ctypes.byref(_t(codes=P + 8, rows=4, block_rows=1)), w, P, 0, 0, None) == 3
    assert f(ctypes.byref(_t(scale=P + 2, rows=4, block_rows=1)), w, P, 0, 0, None) == 3
    assert f(ctypes.byref(_t(scale=None, rows=4, block_rows=1)), w, P, 0, 0, None) == 1
    assert f(ctypes.byref(_t(None, None, 0, 256, 1)), ctypes.byref(_t(None, None)), None, 0, 0, None) == 0
    q = L.nf4_fp8_quantize
    assert q(P, 0, 4, 32, 64, P, P, None) == 4 and q(P, 3, 4, 32, 1, P, P, None) == 2
    assert q(P, 0, 4, 24, 1, P, P, None) == 2 and q(None, 0, 4, 32, 1, P, P, None) == 1
    assert q(P, 0, 4, 32, 1, P + 1, P, None) == 3 and q(None, 0, 0, 32, 1, None, None, None) == 0
    dq = L.nf4_fp8_dequantize
    assert dq(ctypes.byref(_t(block_rows=2)), P, 0, None) == 4
    assert dq(w, P, 5, None) == 2 and dq(w, None, 0, None) == 1


def test_c_abi_validates_norms():
    f, b = nf4.lib().nf4_rmsnorm_fwd, nf4.lib().nf4_rmsnorm_bwd

    def fwd(x=P, xe=1, res=P, re=1, w=P, we=0, rows=4, cols=32, eps=1e-6, h=P, y=P, ye=1, scale=None,
            rstd=None):
        return f(x, xe, res, re, w, we, rows, cols, eps, h, y, ye, scale, rstd, None)

    assert fwd(xe=3) == 2 and fwd(re=2) == 2 and fwd(we=9) == 2 and fwd(ye=4) == 2
    assert fwd(rows=-1) == 2 and fwd(eps=-1.0) == 2 and fwd(cols=24, scale=P) == 2
    assert fwd(x=None) == 1 and fwd(h=None) == 1 and fwd(res=None) == 1 and fwd(y=None) == 1
    assert fwd(x=P + 2) == 3 and fwd(rstd=P + 2) == 3 and fwd(rows=0, x=None) == 0

    need = nf4.lib().nf4_rmsnorm_bwd_workspace(4, 32)
    assert need >= 32 * 4 and nf4.lib().nf4_rmsnorm_bwd_workspace(0, 32) == 0

    def bwd(dy=P, h=P, dh=None, e=1, w=P, we=0, rstd=P, rows=4, cols=32, dx=P, dw=P, ws=P, size=need):
        return b(dy, h, dh, e, w, we, rstd, rows, cols, dx, dw, ws, size, None)

    assert bwd(e=3) == 2 and bwd(rows=-1) == 2 and bwd(size=need - 1) == 2
    assert bwd(dy=None) == 1 and bwd(dw=None) == 1 and bwd(ws=None) == 1
    assert bwd(dh=P + 2) == 3 and bwd(dw=P + 4) == 3 and bwd(cols=0, dw=None) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_valid_calls_without_a_device_report_it():
    L = nf4.lib()
    a, w = ctypes.byref(_t(rows=4, block_rows=1)), ctypes.byref(_t())
    assert L.nf4_fp8_matmul_fwd(a, w, P, 0, 0, None) == 5
    assert L.nf4_fp8_quantize(P, 0, 4, 32, 1, P, P, None) == 5
