"""A transformer's MLP block on the 8-bit operators: the norm adds the residual
and writes the 8-bit operand that the gate and up products read, one kernel takes
both, the activation and its product to the down product's 8-bit operand, and the
stream goes on in 32 bits.

    python examples/fp8_mlp_block.py [hidden] [inner] [tokens]

Trains the norm's weight for a few steps through the frozen block, decodes one
token, and prints losses and the distance to the same block in torch.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dequant_gemm_gb300 as nf4  # noqa: E402
from dequant_gemm_gb300.autograd import FP8GatedMLP, norm_fp8_gated_mlp  # noqa: E402


class FP8MLPBlock(torch.nn.Module):
    """(x, stream) -> (down(silu(gate(n)) * up(n)), stream + x), n the norm of the
    new stream."""

    def __init__(self, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor, eps: float = 1e-6):
        super().__init__()
        self.norm_weight = torch.nn.Parameter(torch.ones(gate.shape[1], device=gate.device))
        self.mlp = FP8GatedMLP(gate, up, down)
        self.eps = eps

    def forward(self, x, stream):
        h, y = norm_fp8_gated_mlp(x, self.norm_weight, *self.mlp.quantized_weights(), residual=stream,
                                  eps=self.eps)
        return y, h


def torch_block(x, stream, norm_weight, gate, up, down, eps=1e-6):
    """The same block in torch's 32-bit arithmetic, nothing rounded to 8 bits."""
    h = stream + x.float()
    n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + eps) * norm_weight
    return torch.nn.functional.linear(
        torch.nn.functional.silu(n @ gate.t()) * (n @ up.t()), down), h


def run(hidden=1024, inner=2816, tokens=512, steps=4, device="cuda:0", quiet=False):
    gen = torch.Generator(device=device).manual_seed(0)
    rand = lambda *s, std=1.0: torch.randn(*s, generator=gen, device=device) * std  # noqa: E731
    gate, up = rand(inner, hidden, std=0.02), rand(inner, hidden, std=0.02)
    down = rand(hidden, inner, std=0.02)
    block = FP8MLPBlock(gate, up, down)
    x, stream = rand(tokens, hidden).bfloat16(), rand(tokens, hidden)
    target = rand(tokens, hidden)

    with torch.no_grad():
        y, h = block(x, stream)
        want, _ = torch_block(x, stream, block.norm_weight, gate, up, down)
        off = float((y.float() - want).norm() / want.norm())

    losses = []
    opt = torch.optim.Adam(block.parameters(), lr=5e-3)
    for _ in range(steps):
        y, h = block(x, stream)
        loss = (h + y.float() - target).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))

    with torch.no_grad():           # one token; the block returns its new stream
        token, _ = block(x[:1], stream[:1])
    status = nf4.nf4_poll_device_status()
    if not quiet:
        print(f"hidden {hidden}, inner {inner}, {tokens} tokens")
        print(f"distance to the 32-bit block: {off:.4f} (relative)")
        print("losses:", " ".join(f"{v:.6f}" for v in losses))
        print(f"one token: {tuple(token.shape)}; device status {status}")
    return off, losses, token, status


if __name__ == "__main__":
    run(*[int(a) for a in sys.argv[1:4]])
