"""Pins of the e4m3 / RMS norm oracle (CPU)."""
import numpy as np
import torch

from oracle import fp8_oracle as o


def test_values_match_torch_bit_for_bit():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(o.VALUES, t, equal_nan=True)
    assert np.nanmax(o.VALUES) == 448.0


def test_round_matches_torch_below_saturation_and_saturates_above():
    g = np.random.default_rng(0)
    x = np.concatenate([g.normal(size=20000) * 2.0 ** g.integers(-14, 9, 20000),
                        (o.VALUES[:126] + o.VALUES[1:127]) / 2,          # every tie
                        o.VALUES[:127], [2.0 ** -10, 2.0 ** -11, 0.0, -0.0]]).astype(np.float32)
    x = x[np.abs(x) <= 448]
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(o.e4m3_round(x), want)
    assert np.array_equal(o.e4m3_round([449.0, 1e30, -1e30, np.nan]), [126, 126, 254, 127])


def test_quantize_blocks():
    x = np.zeros((3, 160), np.float32)
    x[0, :128] = 1.0
    x[0, 128] = -896.0
    x[1, 5] = 2.0 ** -118                              # below the smallest block maximum
    x[2, 130] = np.inf
    codes, scale = o.quantize(x, 1)
    v = o.values(codes, scale, 1)
    assert scale[0, 1] == 2.0 and v[0, 128] == -896.0
    assert abs(v[0, 0] - 1.0) < 1e-7 and scale[1, 0] == 0 and not codes[1].any()
    assert np.isnan(v[2, 128:]).all() and not v[2, :128].any()
    codes, scale = o.quantize(x[:2], 128)
    assert scale.shape == (1, 2) and scale[0, 1] == 2.0


def test_norm_gradients_against_differences():
    g = np.random.default_rng(1)
    x, dy, dh = (g.normal(size=(4, 37)) for _ in range(3))
    w = 1 + 0.1 * g.normal(size=37)

    def loss(x, w):
        return (dy * o.rmsnorm(x, w, 1e-3)[0]).sum() + (dh * x).sum()

    dx, dw = o.rmsnorm_grads(dy, x, w, 1e-3, dh)
    step = 1e-6                                        # central: error O(step^2) + O(eps / step)
    for _ in range(5):
        vx, vw = g.normal(size=x.shape), g.normal(size=w.shape)
        num = (loss(x + step * vx, w) - loss(x - step * vx, w)) / (2 * step)
        assert abs(num - (dx * vx).sum()) <= 1e-7 * (1 + abs(num))
        num = (loss(x, w + step * vw) - loss(x, w - step * vw)) / (2 * step)
        assert abs(num - (dw * vw).sum()) <= 1e-7 * (1 + abs(num))


def test_division_by_448_in_three_roundings_is_exact():
    """q = fl(x r), r = fl(1 / 448); fl(q + fl(x - 448 q) r) is the IEEE quotient
    for every fp32 significand: fp64 holds each exact product and remainder."""
    f32, f64 = np.float32, np.float64
    x = (np.arange(1 << 23, dtype=np.uint32) | 0x3F800000).view(f32)
    r = f32(1) / f32(448)
    q = x * r
    rem = (x.astype(f64) - q.astype(f64) * 448).astype(f32)       # one FMA: exact before its rounding
    # fl(rem r + q): the exact sum needs more than fp64 only in bits far below a half ulp of q
    got = (rem.astype(f64) * f64(r) + q.astype(f64)).astype(f32)
    assert np.array_equal(got, x / f32(448))
