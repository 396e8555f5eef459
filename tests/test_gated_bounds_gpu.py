"""The gated block's and the 4-bit operators' C calls write their outputs and
nothing beside them, and what lies beside their inputs does not matter (as
tests/test_operand_bounds_gpu.py for the others)."""
import ctypes
import random

import pytest
import torch

import dequant_gemm_gb300 as nf4
from tests.test_operand_bounds_gpu import Buffers, call, rand, same, size

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8, F32, BF16, F16 = torch.float8_e4m3fn, torch.float32, torch.bfloat16, torch.float16
ELEM = nf4.ELEM


def fp8_in(b, q):
    return ctypes.byref(nf4.nf4_fp8_tensor(b.put(q.codes), b.put(q.scale), q.rows, q.cols, q.block_rows))


def operands(rng, seed):
    M, N, K = size(rng, 1, 700), size(rng, 16, 1500, 16), size(rng, 16, 1500, 16)
    ws = [nf4.nf4_fp8_quantize(rand(N, K, seed=seed + i, std=0.02), block_rows=128) for i in (1, 2)]
    return M, N, K, ws


@pytest.mark.parametrize("seed", range(24))
def test_gated_forward(seed):
    rng, b = random.Random(seed), Buffers()
    M, N, K, (wg, wu) = operands(rng, seed)
    out, save, name = rng.choice([F8, F8, BF16, F32]), rng.random() < 0.5, rng.choice(sorted(nf4.ACTIVATIONS))
    x = nf4.nf4_fp8_quantize(rand(M, K, seed=seed))
    want, g, u = nf4.nf4_fp8_gated_fwd(x, wg, wu, activation=name, out_dtype=out, save=save)
    at, y = b.room((M, N), out)
    at_s, s = b.room((M, -(-N // 128)), F32)
    at_g, G = b.room((M, N), BF16)
    at_u, U = b.room((M, N), BF16)
    call("nf4_fp8_gated_fwd", fp8_in(b, x), fp8_in(b, wg), fp8_in(b, wu), nf4.ACTIVATIONS[name], at, ELEM.get(out, 0),
         at_s if out == F8 else None, at_g if save else None, at_u if save else None)
    assert b.intact()
    assert same(y, want.codes if out == F8 else want) and (out != F8 or same(s, want.scale))
    assert not save or same(G, g) and same(U, u)


@pytest.mark.parametrize("seed", range(12))
def test_gated_gradients(seed):
    rng, b = random.Random(seed), Buffers()
    M, N, dt = size(rng, 1, 700), size(rng, 16, 3000, 16), rng.choice([F32, BF16, F16])
    dy, g, u = rand(M, N, seed=seed, dtype=dt), *(rand(M, N, seed=seed + i, dtype=BF16) for i in (1, 2))
    want = nf4.nf4_fp8_gated_bwd(dy, g, u)
    out = [b.room(*a) for _ in range(2) for a in (((M, N), F8), ((M, -(-N // 128)), F32))]
    call("nf4_fp8_gated_bwd", b.put(dy), ELEM[dt], b.put(g), b.put(u), M, N, 0, *(at for at, _ in out))
    assert b.intact()
    assert all(same(t, w) for (_, t), w in zip(out, (want[0].codes, want[0].scale, want[1].codes, want[1].scale)))


@pytest.mark.parametrize("seed", range(24))
def test_gated_input_gradient(seed):
    rng, b = random.Random(seed), Buffers()
    M, N, K, (wg, wu) = operands(rng, seed)
    out, add = rng.choice([F32, BF16]), rng.random() < 0.5
    dg, du = (nf4.nf4_fp8_quantize(rand(M, N, seed=seed + i)) for i in (3, 4))
    before = rand(M, K, seed=seed + 2, dtype=out)
    want = nf4.nf4_fp8_gated_bwd_dx(dg, du, wg, wu, out=before.clone(), accumulate=add)
    at, y = b.room((M, K), out, before)
    call("nf4_fp8_gated_bwd_dx", fp8_in(b, dg), fp8_in(b, du), fp8_in(b, wg), fp8_in(b, wu), at, ELEM[out], int(add))
    assert b.intact() and same(y, want)


@pytest.mark.parametrize("seed", range(40))
def test_int4(seed):
    rng, b = random.Random(seed), Buffers()
    group, zero = rng.choice([32, 64, 128]), rng.random() < 0.5
    M, N, K = size(rng, 1, 60), size(rng, 1, 600), size(rng, group, 6000, group)
    xt, dt = rng.choice([BF16, F16]), rng.choice([F32, BF16, F16])
    ws = [nf4.nf4_int4_quantize(rand(N, K, seed=seed + i, std=0.02), group=group, zero_point=zero) for i in (1, 2)]
    x = rand(M, K, seed=seed, dtype=xt)

    def put(w):
        return ctypes.byref(nf4.nf4_int4_weight(b.put(w.codes), b.put(w.scale), b.put(w.zero), N, K, group, ELEM[BF16]))

    want = nf4.nf4_int4_matmul_fwd(x, ws[0], out_dtype=dt)
    at, y = b.room((M, N), dt)
    call("nf4_int4_matmul_fwd", b.put(x), ELEM[xt], M, put(ws[0]), at, ELEM[dt], 0)
    assert b.intact() and same(y, want)
    want = nf4.nf4_int4_gated_fwd(x, *ws, out_dtype=dt)
    at, y = b.room((M, N), dt)
    call("nf4_int4_gated_fwd", b.put(x), ELEM[xt], M, put(ws[0]), put(ws[1]), 0, at, ELEM[dt])
    assert b.intact() and same(y, want)
    at, v = b.room((N, K), dt)
    call("nf4_int4_dequantize", put(ws[0]), at, ELEM[dt])
    assert b.intact() and same(v, nf4.nf4_int4_dequantize(ws[0], out_dtype=dt))
    w = rand(N, K, seed=seed + 1, std=0.02)
    (ac, c), (as_, s), (az, z) = (b.room(*a) for a in (((N, K // 2), torch.uint8), ((N, K // group), BF16),
                                                       ((N, K // group), torch.uint8)))
    call("nf4_int4_quantize", b.put(w), 0, N, K, group, ELEM[BF16], ac, as_, az if zero else None)
    assert b.intact() and same(c, ws[0].codes) and same(s, ws[0].scale) and (not zero or same(z, ws[0].zero))
