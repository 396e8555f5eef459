"""The 8-bit operators and the norm in a chain, each launched programmatically
behind the one before: back to back, and captured in a CUDA graph replayed on
new inputs, every output has the bits of the same calls with a synchronisation
after each. A kernel that read before its predecessor had written would not."""
import pytest
import torch

import dequant_gemm_gb300 as nf4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8, F32, BF16 = torch.float8_e4m3fn, torch.float32, torch.bfloat16
HIDDEN, INNER = 576, 1040      # neither in whole blocks of 128


def normal(*shape, seed, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).to(DEV)


def chain(s, wait):
    """All outputs of a pass over s, the weights quantized within it."""
    out = []

    def did(*tensors):
        out.extend(t for t in tensors if t is not None)
        if wait:
            torch.cuda.synchronize()

    up = nf4.nf4_fp8_quantize(s["up"], block_rows=128)
    did(up.codes, up.scale)
    q, h, r = nf4.nf4_rmsnorm_fwd(s["x"], s["norm"], s["stream"], out_dtype=F8, save_rstd=True)
    did(q.codes, q.scale, h, r)
    y = nf4.nf4_fp8_matmul_fwd(q, up, out_dtype=BF16)
    did(y)
    q = nf4.nf4_fp8_quantize(y)
    did(q.codes, q.scale)
    down = nf4.nf4_fp8_quantize(s["down"], block_rows=128)
    did(down.codes, down.scale)
    z = nf4.nf4_fp8_matmul_fwd(q, down)
    did(z)
    n, h2, r2 = nf4.nf4_rmsnorm_fwd(z, s["norm"], h, out_dtype=BF16, save_rstd=True, out_h=h.clone())
    did(n, h2, r2)
    four = nf4.nf4_quantize(s["four"])
    did(four.codes, four.absmax_q, four.absmax_scale)
    n = nf4.nf4_matmul_fwd(n, four, out_dtype=BF16)
    did(n)
    d = nf4.nf4_fp8_quantize(n)
    did(d.codes, d.scale)
    d = nf4.nf4_fp8_matmul_bwd_dx(d, down)
    did(d)
    q = nf4.nf4_fp8_quantize(d)
    did(q.codes, q.scale)
    d = nf4.nf4_fp8_matmul_bwd_dx(q, up)
    did(d)
    dx, dw = nf4.nf4_rmsnorm_bwd(d, h2, s["norm"], r2, dh=z)
    did(dx, dw)
    did(nf4.nf4_fp8_dequantize(nf4.nf4_fp8_quantize(dx)))
    return out


def bits(t):
    return t.view(torch.uint8) if t.dtype == F8 else t


def inputs(M, seed):
    return {"x": normal(M, HIDDEN, seed=seed, dtype=BF16), "stream": normal(M, HIDDEN, seed=seed + 1),
            "norm": 1 + normal(HIDDEN, seed=seed + 2, std=0.1), "up": normal(INNER, HIDDEN, seed=seed + 3, std=0.02),
            "down": normal(HIDDEN, INNER, seed=seed + 4, std=0.02), "four": normal(HIDDEN, HIDDEN, seed=seed + 5, std=0.02)}


@pytest.mark.parametrize("M", [1, 40, 300])
def test_chain_back_to_back_and_in_a_graph(M):
    batches = [inputs(M, 10 * k) for k in range(1, 5)]
    want = [chain(s, wait=True) for s in batches]
    for s, ref in zip(batches, want):
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(chain(s, wait=False), ref))
    static = {k: v.clone() for k, v in batches[0].items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(static, wait=False)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(static, wait=False)
    for _ in range(3):
        for s, ref in zip(batches, want):
            for k, v in s.items():
                static[k].copy_(v)
            graph.replay()
            graph.replay()               # the next pass's kernels right behind the last one's
            assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, ref))
    assert nf4.nf4_poll_device_status() == 0
