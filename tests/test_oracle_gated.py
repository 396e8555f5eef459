"""Pins of the gated block's and the 4-bit format's oracle."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import gated_oracle as o


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
def test_activation(name):
    g = np.linspace(-12, 12, 4001)
    f, slope = o.act(g, name)
    t = torch.from_numpy(g)
    want = torch.nn.functional.silu(t) if name == "silu" else torch.nn.functional.gelu(t, approximate="tanh")
    assert np.allclose(f, want.numpy(), rtol=1e-13, atol=1e-15)
    # central differences: the third derivative is below 2 everywhere, so the
    # error is below h^2 / 3 and the rounding 2e-15 / h
    h = 1e-5
    diff = (o.act(g + h, name)[0] - o.act(g - h, name)[0]) / (2 * h)
    assert np.abs(diff - slope).max() < h * h + 2e-15 / h * 12
    # the same by sigma(p(g)), which the kernels use
    p, dp = o.exponent(g, name)
    s = 1 / (1 + np.exp(-p))
    assert np.allclose(g * s, f, rtol=1e-11, atol=1e-13)
    assert np.allclose(s + g * s * (1 - s) * dp, slope, rtol=1e-11, atol=1e-13)


@pytest.mark.parametrize("zero", [True, False])
@pytest.mark.parametrize("scale", ["bf16", "f16"])
def test_codes_are_the_nearest_of_the_exact_quotient(zero, scale):
    rng = np.random.default_rng(3)
    w = (rng.standard_normal((6, 64)) * 0.02).astype(np.float32)
    w[1, :32], w[2, 5] = 0, 0.3
    w[3] = np.abs(w[3])                       # one-sided groups
    q, s, z = o.int4_quantize(w, 32, zero, scale)
    for i in range(6):
        for k in range(64):
            si, zi = Fraction(float(s[i, k // 32])), int(z[i, k // 32])
            if si == 0:
                assert q[i, k] == zi
                continue
            quotient = Fraction(float(w[i, k])) / si
            code = int(q[i, k]) - zi
            inside = 0 < q[i, k] < 15
            # the fp32 quotient is off by 2^-24 of 15 at most
            assert not inside or abs(quotient - code) <= Fraction(1, 2) + Fraction(15, 1 << 24)
            assert inside or abs(quotient) >= abs(code) - Fraction(1, 2) - Fraction(15, 1 << 24)
    v = o.int4_values(o.int4_pack(q), s, z if zero else None)
    # within half a step, plus what the clamp cuts off: the scale's rounding moves
    # the range's ends by 15 (7) steps of half an ulp, the zero point by half a step
    u = 2.0 ** -8 if scale == "bf16" else 2.0 ** -11
    step = np.repeat(s.astype(np.float64), 32, 1)
    assert (np.abs(v - w) <= step * ((1.0 if zero else 0.5) + 15 * u) + 1e-9).all()
    assert (v[1, :32] == 0).all()


def test_packing_puts_the_even_element_high():
    q = np.arange(16, dtype=np.uint8).reshape(1, 16)
    assert o.int4_pack(q)[0].tolist() == [0x01, 0x23, 0x45, 0x67, 0x89, 0xab, 0xcd, 0xef]
    s = np.array([[2.0]])
    assert o.int4_values(o.int4_pack(q), s, None)[0].tolist() == [2.0 * (i - 8) for i in range(16)]
    assert o.int4_values(o.int4_pack(q), s, np.array([[3]], np.uint8))[0, 5] == 4.0
