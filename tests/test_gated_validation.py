"""Refusals of the gated block and of the 4-bit weights in groups: the Python
checks on CPU tensors, and the C entry points' host-side validation."""
import ctypes

import pytest
import torch

import dequant_gemm_gb300 as nf4

P = 1 << 20   # a fake aligned address, never dereferenced by validation
F8, BF16 = torch.float8_e4m3fn, torch.bfloat16


def act(rows=4, cols=256):
    return nf4.alloc_fp8(rows, cols, "cpu")


def weight(rows=32, cols=256):
    return nf4.alloc_fp8(rows, cols, "cpu", block_rows=128)


def int4(rows=32, cols=256, group=128, zero=True, scale=BF16, device="cpu"):
    shape = (rows, cols // group)
    return nf4.Int4Weight(torch.zeros(rows, cols // 2, dtype=torch.uint8, device=device),
                          torch.zeros(shape, dtype=scale, device=device),
                          torch.zeros(shape, dtype=torch.uint8, device=device) if zero else None)


def test_gated_forward_refuses():
    f, x, g, u = nf4.nf4_fp8_gated_fwd, act(), weight(), weight()
    for args, kw, match in (((torch.zeros(4, 256), g, u), {}, "FP8Tensor"), ((x, g, torch.zeros(32, 256)), {}, "FP8Tensor"),
                            ((act(cols=128), g, u), {}, "must be"), ((x, g, weight(48)), {}, "same shape"),
                            ((x, g, weight(32, 128)), {}, "same shape"), ((x, act(32), u), {}, "block_rows"),
                            ((x, g, act(32)), {}, "block_rows"), ((g, g, u), {}, "block_rows"),
                            ((x, weight(24), weight(24)), {}, "multiple of 16"),
                            ((nf4.FP8Tensor(x.codes, x.scale[:, :1].contiguous()), g, u), {}, "shape"),
                            ((x, g, nf4.FP8Tensor(u.codes.view(torch.uint8), u.scale, 128)), {}, "float8"),
                            ((x, g, u), dict(activation="relu"), "activation"),
                            ((x, g, u), dict(activation=0), "activation"),
                            ((x, g, u), dict(out_dtype=torch.float16), "output"),
                            ((x, g, nf4.alloc_fp8(32, 256, "meta", 128)), {}, "expected cpu"),
                            ((x, g, u), {}, "CUDA device")):
        with pytest.raises(ValueError, match=match):
            f(*args, **kw)


def test_gated_backward_refuses():
    f = nf4.nf4_fp8_gated_bwd
    d, g, u = torch.zeros(4, 32), *(torch.zeros(4, 32, dtype=BF16) for _ in range(2))
    for args, kw, match in (((d.int(), g, u), {}, "dy must be"), ((d, g.float(), u), {}, "g must be"),
                            ((d, g, u[:2]), {}, "shape"), ((d[:, ::2], g[:, ::2], u[:, ::2]), {}, "contiguous"),
                            ((d[0], g[0], u[0]), {}, "2-D"),
                            ((d[:, :24].contiguous(), g[:, :24].contiguous(), u[:, :24].contiguous()), {}, "multiple of 16"),
                            ((d, g, u), dict(activation="gelu"), "activation"),
                            ((d, g, u.to("meta")), {}, "expected cpu"), ((d, g, u), {}, "CUDA device")):
        with pytest.raises(ValueError, match=match):
            f(*args, **kw)
    f, dg, w = nf4.nf4_fp8_gated_bwd_dx, act(4, 32), weight()
    for args, kw, match in (((act(), dg, w, w), {}, "must be"), ((dg, act(), w, w), {}, "must be"),
                            ((dg, act(5, 32), w, w), {}, "same rows"), ((dg, dg, w, weight(48)), {}, "same shape"),
                            ((dg, dg, act(32), w), {}, "block_rows"), ((dg, dg, w, w), dict(accumulate=True), "accumulate"),
                            ((dg, dg, w, w), dict(out=torch.zeros(4, 255)), "shape"),
                            ((dg, dg, w, w), dict(out=3), "tensor"),
                            ((dg, dg, w, w), dict(out_dtype=F8), "float32 or bfloat16"), ((dg, dg, w, w), {}, "CUDA device")):
        with pytest.raises(ValueError, match=match):
            f(*args, **kw)


def test_int4_refuses():
    f, w = nf4.nf4_int4_quantize, torch.zeros(4, 256)
    for args, kw, match in (((w.int(),), {}, "float32"), ((w[0],), {}, "2-D"), ((w[:, ::2],), {}, "contiguous"),
                            ((w,), dict(group=16), "group"), ((w[:, :96].contiguous(),), {}, "multiple of the group"),
                            ((w,), dict(scale_dtype=torch.float32), "scale_dtype"),
                            ((w,), dict(out=int4(4, 128)), "asked for"), ((w,), dict(out=int4(4, group=64)), "asked for"),
                            ((w,), dict(out=int4(4, zero=False)), "asked for"),
                            ((w,), dict(out=int4(4, scale=torch.float16)), "asked for"), ((w,), {}, "CUDA device")):
        with pytest.raises(ValueError, match=match):
            f(*args, **kw)
    for call in (nf4.nf4_int4_dequantize, lambda w: nf4.nf4_int4_matmul_fwd(torch.zeros(2, 256, dtype=BF16), w),
                 lambda w: nf4.nf4_int4_gated_fwd(torch.zeros(2, 256, dtype=BF16), int4(), w)):
        good = int4()
        for bad, match in ((torch.zeros(2), "Int4Weight"), (nf4.Int4Weight(good.codes.to(torch.int8), good.scale), "uint8"),
                           (nf4.Int4Weight(good.codes, good.scale.float()), "float16 or bfloat16"),
                           (nf4.Int4Weight(good.codes, good.scale[:3]), "shape"),
                           (nf4.Int4Weight(good.codes, good.scale[0]), "2-D"),
                           (nf4.Int4Weight(good.codes, good.scale, good.zero[:, :1].contiguous()), "shape"),
                           (nf4.Int4Weight(good.codes, good.scale, good.zero.int()), "uint8"),
                           (nf4.Int4Weight(good.codes, torch.zeros(32, 1, dtype=BF16)), "group must be"),
                           (nf4.Int4Weight(good.codes, torch.zeros(32, 3, dtype=BF16)), "columns in 3 groups"),
                           (nf4.Int4Weight(good.codes, good.scale.to("meta")), "expected cpu"), (good, "CUDA device")):
            with pytest.raises(ValueError, match=match):
                call(bad)
    x, w = torch.zeros(2, 256, dtype=BF16), int4()
    for kw, match in ((dict(X=x.float()), "bfloat16 or float16"), (dict(X=x[:, :128]), "contiguous"),
                      (dict(X=x[0]), "must be"), (dict(X=x.view(4, 128)), "must be"),
                      (dict(out_dtype=torch.int8), "output"), (dict(out=torch.zeros(2, 31)), "shape"),
                      (dict(accumulate=True), "accumulate"), (dict(out=torch.zeros(2, 32, device="meta")), "expected cpu")):
        with pytest.raises(ValueError, match=match):
            nf4.nf4_int4_matmul_fwd(**{"X": x, "w": w, **kw})
    for up, kw, match in ((int4(48), {}, "same shape"), (int4(group=64), {}, "same shape"),
                          (int4(scale=torch.float16), {}, "scale type"), (w, dict(activation="tanh"), "activation"),
                          (w, dict(out_dtype=torch.int8), "output")):
        with pytest.raises(ValueError, match=match):
            nf4.nf4_int4_gated_fwd(x, w, up, **kw)


def test_int4_products_refuse_longer_rows():
    K = 262144 + 128
    x, w = torch.zeros(1, K, dtype=BF16), int4(1, K)
    for call in (nf4.nf4_int4_matmul_fwd, lambda x, w: nf4.nf4_int4_gated_fwd(x, w, w)):
        with pytest.raises(ValueError, match="262144 at most"):
            call(x, w)
    assert nf4.lib().nf4_int4_matmul_fwd(P, 1, 1, w4(1, K), P, 0, 0, None) == 2
    assert nf4.lib().nf4_int4_gated_fwd(P, 1, 1, w4(1, K), w4(1, K), 0, P, 0, None) == 2


def q8(rows, cols, block_rows=1, codes=P, scale=P):
    return ctypes.byref(nf4.nf4_fp8_tensor(codes, scale, rows, cols, block_rows))


def test_c_gated_validation():
    L = nf4.lib()

    def fwd(X=None, g=None, u=None, act=0, y=P, elem=1, scale=None, G=None, U=None):
        return L.nf4_fp8_gated_fwd(X or q8(4, 256), g or q8(32, 256, 128), u or q8(32, 256, 128), act, y, elem, scale,
                                   G, U, None)

    assert fwd(act=2) == 2 and fwd(act=-1) == 2 and fwd(elem=2) == 2
    assert fwd(y=None) == 1 and fwd(G=P) == 1 and fwd(U=P) == 1 and fwd(X=q8(4, 256, codes=None)) == 1
    assert fwd(g=q8(32, 256, 1)) == 4 and fwd(u=q8(32, 256, 1)) == 4 and fwd(X=q8(4, 256, 128)) == 4
    assert fwd(g=q8(48, 256, 128)) == 2 and fwd(X=q8(4, 128)) == 2 and fwd(X=q8(-1, 256)) == 2
    assert fwd(y=P + 8) == 3 and fwd(scale=P + 2) == 3 and fwd(G=P + 8, U=P) == 3 and fwd(G=P, U=P + 4) == 3
    assert fwd(u=q8(32, 256, 128, codes=P + 4)) == 3
    assert fwd(X=q8(0, 256, codes=None), y=None) == 0
    assert L.nf4_fp8_gated_fwd(None, None, None, 0, P, 0, None, None, None, None) == 1

    def bwd(elem=0, rows=4, cols=32, act=0, dy=P, g=P, u=P, dg=P, sg=P, du=P, su=P):
        return L.nf4_fp8_gated_bwd(dy, elem, g, u, rows, cols, act, dg, sg, du, su, None)

    assert bwd(elem=3) == 2 and bwd(cols=24) == 2 and bwd(rows=-1) == 2 and bwd(act=5) == 2
    for name in ("dy", "g", "u", "dg", "sg", "du", "su"):
        assert bwd(**{name: None}) == 1 and bwd(**{name: P + 2}) == 3
    assert bwd(rows=0, dy=None) == 0

    def dx(dg=None, du=None, g=None, u=None, out=P, elem=0, flags=0):
        return L.nf4_fp8_gated_bwd_dx(dg or q8(4, 32), du or q8(4, 32), g or q8(32, 256, 128), u or q8(32, 256, 128), out,
                                      elem, flags, None)

    assert dx(elem=2) == 2 and dx(flags=2) == 2 and dx(du=q8(5, 32)) == 2 and dx(dg=q8(4, 48)) == 2
    assert dx(u=q8(32, 128, 128)) == 2 and dx(u=q8(32, 256, 1)) == 4 and dx(du=q8(4, 32, 128)) == 4
    assert dx(out=None) == 1 and dx(out=P + 4) == 3 and dx(du=q8(4, 32, codes=None)) == 1
    assert dx(dg=q8(0, 32), du=q8(0, 32), out=None) == 0


def w4(rows=32, cols=256, group=128, elem=1, codes=P, scale=P, zero=None):
    return ctypes.byref(nf4.nf4_int4_weight(codes, scale, zero, rows, cols, group, elem))


def test_c_int4_validation():
    L = nf4.lib()

    def quant(w=P, elem=0, rows=4, cols=256, group=128, se=1, codes=P, scale=P, zero=None):
        return L.nf4_int4_quantize(w, elem, rows, cols, group, se, codes, scale, zero, None)

    assert quant(group=16) == 4 and quant(group=256) == 4 and quant(elem=3) == 2 and quant(se=0) == 2
    assert quant(cols=192) == 2 and quant(rows=-1) == 2 and quant(w=None) == 1 and quant(codes=None) == 1
    assert quant(scale=None) == 1 and quant(w=P + 8) == 3 and quant(codes=P + 8) == 3 and quant(scale=P + 1) == 3
    assert quant(rows=0, w=None) == 0 and quant(cols=0, w=None) == 0

    assert L.nf4_int4_dequantize(None, P, 0, None) == 1 and L.nf4_int4_dequantize(w4(), P, 4, None) == 2
    assert L.nf4_int4_dequantize(w4(), None, 0, None) == 1 and L.nf4_int4_dequantize(w4(), P + 4, 0, None) == 3

    def fwd(X=P, elem=1, M=4, w=None, Y=P, ye=0, flags=0):
        return L.nf4_int4_matmul_fwd(X, elem, M, w or w4(), Y, ye, flags, None)

    assert fwd(elem=0) == 2 and fwd(M=-1) == 2 and fwd(M=1 << 31) == 2 and fwd(ye=3) == 2 and fwd(flags=4) == 2
    assert fwd(w=w4(group=48)) == 4 and fwd(w=w4(elem=0)) == 2 and fwd(w=w4(cols=200)) == 2
    assert fwd(X=None) == 1 and fwd(Y=None) == 1 and fwd(w=w4(codes=None)) == 1 and fwd(w=w4(scale=None)) == 1
    assert fwd(X=P + 8) == 3 and fwd(Y=P + 2) == 3 and fwd(Y=P + 1, ye=1) == 3 and fwd(w=w4(codes=P + 8)) == 3
    assert fwd(M=0, X=None) == 0 and L.nf4_int4_matmul_fwd(P, 1, 4, None, P, 0, 0, None) == 1

    def gated(g=None, u=None, act=0):
        return L.nf4_int4_gated_fwd(P, 1, 4, g or w4(), u or w4(), act, P, 0, None)

    assert gated(act=9) == 2 and gated(u=w4(rows=33)) == 2 and gated(u=w4(group=64)) == 2 and gated(u=w4(elem=2)) == 2
    assert gated(u=w4(codes=None)) == 1 and gated(u=w4(scale=P + 1)) == 3
    assert L.nf4_int4_gated_fwd(P, 1, 4, w4(), None, 0, P, 0, None) == 1
