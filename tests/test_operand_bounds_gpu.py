"""The 8-bit operators and the norm write their outputs and nothing beside them,
and what lies beside their inputs does not matter: each C call runs on operands
in the middle of larger buffers, outputs among a pattern that has to survive,
inputs among NaN bytes (0xff is NaN in fp32, bf16, fp16 and e4m3), and gives the bits
of the Python call on tensors of their own."""
import ctypes
import random

import pytest
import torch

import dequant_gemm_gb300 as nf4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8, F32, BF16, F16 = torch.float8_e4m3fn, torch.float32, torch.bfloat16, torch.float16
ELEM = nf4.ELEM
PAD = 4096                  # bytes on either side, a multiple of 16


def rand(*shape, seed, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).to(DEV)


class Buffers:
    """Operands inside larger buffers."""

    def __init__(self):
        self.checks = []

    def put(self, t):
        """An input: a copy of t among NaN bytes."""
        if t is None:
            return None
        raw = torch.full((t.nbytes + 2 * PAD,), 0xff, dtype=torch.uint8, device=DEV)
        raw[PAD:PAD + t.nbytes] = t.contiguous().view(-1).view(torch.uint8)
        self.checks.append((raw, t.nbytes, 0xff))
        return raw.data_ptr() + PAD

    def room(self, shape, dtype, init=None):
        """An output: (address, tensor), among a pattern."""
        n = torch.empty(shape, dtype=dtype, device="meta").nbytes
        raw = torch.full((n + 2 * PAD,), 0xa5, dtype=torch.uint8, device=DEV)
        if init is not None:
            raw[PAD:PAD + n] = init.contiguous().view(-1).view(torch.uint8)
        self.checks.append((raw, n, 0xa5))
        return raw.data_ptr() + PAD, raw[PAD:PAD + n].view(dtype).view(shape)

    def intact(self):
        torch.cuda.synchronize()
        return all(bool((raw[:PAD] == p).all() and (raw[PAD + n:] == p).all()) for raw, n, p in self.checks)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def call(name, *args):
    status = getattr(nf4.lib(), name)(*args, torch.cuda.current_stream().cuda_stream)
    assert status == 0


def size(rng, lo, hi, step=1):
    return max(step, int(round(lo * (hi / lo) ** rng.random() / step)) * step)


@pytest.mark.parametrize("seed", range(24))
def test_products(seed):
    rng, b = random.Random(seed), Buffers()
    M, N, K = size(rng, 1, 700), size(rng, 16, 1500, 16), size(rng, 16, 1500, 16)
    dx, out, add = rng.random() < 0.5, rng.choice([F32, BF16]), rng.random() < 0.5
    red, cols = (N, K) if dx else (K, N)
    a = nf4.nf4_fp8_quantize(rand(M, red, seed=seed))
    w = nf4.nf4_fp8_quantize(rand(N, K, seed=seed + 1, std=0.02), block_rows=128)
    before = rand(M, cols, seed=seed + 2, dtype=out)
    name = "nf4_fp8_matmul_bwd_dx" if dx else "nf4_fp8_matmul_fwd"
    want = getattr(nf4, name)(a, w, out=before.clone(), accumulate=add)
    at, y = b.room((M, cols), out, before)
    call(name, ctypes.byref(nf4.nf4_fp8_tensor(b.put(a.codes), b.put(a.scale), M, red, 1)),
         ctypes.byref(nf4.nf4_fp8_tensor(b.put(w.codes), b.put(w.scale), N, K, 128)), at, ELEM[out], int(add))
    assert b.intact() and same(y, want)


@pytest.mark.parametrize("seed", range(12))
def test_quantizer(seed):
    rng, b = random.Random(seed), Buffers()
    rows, cols, block = size(rng, 1, 900), size(rng, 16, 3000, 16), rng.choice([1, 128])
    dtype, back = rng.choice([F32, BF16, F16]), rng.choice([F32, BF16, F16])
    x = rand(rows, cols, seed=seed, dtype=dtype)
    want = nf4.nf4_fp8_quantize(x, block_rows=block)
    at, codes = b.room((rows, cols), F8)
    sat, scale = b.room(want.scale.shape, F32)
    call("nf4_fp8_quantize", b.put(x), ELEM[dtype], rows, cols, block, at, sat)
    assert b.intact() and same(codes, want.codes) and same(scale, want.scale)
    at, v = b.room((rows, cols), back)
    call("nf4_fp8_dequantize", ctypes.byref(nf4.nf4_fp8_tensor(b.put(want.codes), b.put(want.scale), rows, cols, block)),
         at, ELEM[back])
    assert b.intact() and same(v, nf4.nf4_fp8_dequantize(want, out_dtype=back))


LENGTHS = [1, 7, 24, 257, 528, 1023, 2048, 3584, 5001, 5384, 8177, 8187, 8200, 12000, 16379, 16392, 20000, 33001]


@pytest.mark.parametrize("cols", LENGTHS)
@pytest.mark.parametrize("x_dtype, res_dtype, out", [(F32, None, F32), (BF16, F32, F8), (F16, F16, BF16), (BF16, None, BF16),
                                                     (F32, F32, F16)])
def test_norm(cols, x_dtype, res_dtype, out):
    rows, b = 1 + cols % 13, Buffers()
    if out == F8 and cols % 16:
        out = BF16
    x, w = rand(rows, cols, seed=cols, dtype=x_dtype), 1 + rand(cols, seed=2, std=0.1)
    res = None if res_dtype is None else rand(rows, cols, seed=3, dtype=res_dtype)
    y, h, r = nf4.nf4_rmsnorm_fwd(x, w, res, out_dtype=out, save_rstd=True)
    yat, y2 = b.room((rows, cols), out)
    hat, h2 = (None, None) if res is None else b.room((rows, cols), res_dtype)
    sat, s2 = b.room((rows, -(-cols // 128)), F32) if out == F8 else (None, None)
    rat, r2 = b.room((rows,), F32)
    call("nf4_rmsnorm_fwd", b.put(x), ELEM[x_dtype], b.put(res), 0 if res is None else ELEM[res_dtype], b.put(w), ELEM[F32],
         rows, cols, 1e-6, hat, yat, 0 if out == F8 else ELEM[out], sat, rat)
    assert b.intact() and same(r2, r) and (res is None or same(h2, h))
    assert same(y2, y.codes) and same(s2, y.scale) if out == F8 else same(y2, y)


@pytest.mark.parametrize("cols", LENGTHS)
@pytest.mark.parametrize("dtype, w_dtype", [(F32, F32), (BF16, F32), (F16, F16)])
@pytest.mark.parametrize("rows", [1, 6, 333])
def test_norm_gradients(rows, cols, dtype, w_dtype):
    b = Buffers()
    h, dy, dh = (rand(rows, cols, seed=s, dtype=dtype) for s in (1, 2, 3))
    dh = dh if cols % 3 else None
    w = (1 + rand(cols, seed=4, std=0.1)).to(w_dtype)
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    dx, dw = nf4.nf4_rmsnorm_bwd(dy, h, w, rstd, dh=dh)
    n = nf4.lib().nf4_rmsnorm_bwd_workspace(rows, cols)
    xat, dx2 = b.room((rows, cols), dtype)
    wat, dw2 = b.room((cols,), w_dtype)
    wsat, _ = b.room((n,), torch.uint8)
    call("nf4_rmsnorm_bwd", b.put(dy), b.put(h), b.put(dh), ELEM[dtype], b.put(w), ELEM[w_dtype], b.put(rstd), rows, cols,
         xat, wat, wsat, n)
    assert b.intact() and same(dx2, dx) and same(dw2, dw)
