"""Tensors that a call writes into (out=, out_h=) count as modified, as torch's
own in-place operations do: a backward pass that saved one raises instead of
using the new values."""
import pytest
import torch

import dequant_gemm_gb300 as nf4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rand(*shape, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(sum(shape))).to(dtype).to(DEV)


def calls():
    W, X = rand(128, 256), rand(20, 256, dtype=torch.bfloat16)
    q, q8, w8 = nf4.nf4_quantize(W), nf4.nf4_fp8_quantize(X), nf4.nf4_fp8_quantize(W, block_rows=128)
    d, d8 = rand(20, 128, dtype=torch.bfloat16), nf4.nf4_fp8_quantize(rand(20, 128))
    one = torch.ones(256, device=DEV)
    y, x = torch.zeros(20, 128, device=DEV), torch.zeros(20, 256, device=DEV)
    return {
        "quantize": ([q.codes, q.absmax_q, q.absmax_scale], lambda: nf4.nf4_quantize(W, out=q)),
        "dequantize": ([W2 := rand(128, 256)], lambda: nf4.nf4_dequantize(q, out=W2)),
        "fwd": ([y], lambda: nf4.nf4_matmul_fwd(X, q, out=y, accumulate=True)),
        "group": ([y, z := y.clone()], lambda: nf4.nf4_matmul_fwd_group(X, [q, q], outs=[y, z])),
        "dx": ([x], lambda: nf4.nf4_matmul_bwd_dx(d, q, out=x)),
        "fp8_quantize": ([q8.codes, q8.scale], lambda: nf4.nf4_fp8_quantize(X, out=q8)),
        "fp8_dequantize": ([x], lambda: nf4.nf4_fp8_dequantize(q8, out=x)),
        "fp8_fwd": ([y], lambda: nf4.nf4_fp8_matmul_fwd(q8, w8, out=y)),
        "fp8_dx": ([x], lambda: nf4.nf4_fp8_matmul_bwd_dx(d8, w8, out=x, accumulate=True)),
        "norm": ([x], lambda: nf4.nf4_rmsnorm_fwd(X, one, x, out_h=x)),
    }


@pytest.mark.parametrize("name", ["quantize", "dequantize", "fwd", "group", "dx", "fp8_quantize", "fp8_dequantize",
                                  "fp8_fwd", "fp8_dx", "norm"])
def test_version_counts(name):
    tensors, call = calls()[name]
    before = [t._version for t in tensors]
    call()
    assert all(t._version > v for t, v in zip(tensors, before))


def test_a_saved_stream_changed_in_place_is_noticed():
    s = rand(4, 256).requires_grad_()
    stream = s * 1.0
    loss = stream.square().sum()                  # saves the stream
    with torch.no_grad():
        nf4.nf4_rmsnorm_fwd(rand(4, 256), torch.ones(256, device=DEV), stream, out_h=stream)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inference_tensors_are_written_anywhere():
    with torch.inference_mode():
        stream, x, w = rand(4, 256), rand(4, 256), torch.ones(256, device=DEV)
        nf4.nf4_rmsnorm_fwd(x, w, stream, out_h=stream)
    nf4.nf4_rmsnorm_fwd(x, w, stream, out_h=stream)
