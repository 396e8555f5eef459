// The gradients of the gated block's product (gated.cuh), in 8 bits for the two
// products that make the input gradient of them (fp8_gemm.cu):
//   dG = dY U act'(G), dU = dY act(G),
//   act'(g) = s + g s (1 - s) p'(g), s = sigma(p(g)), p'(g) = c0 + 3 c1 g^2
#include "gated.cuh"

namespace nf4 {
namespace {

// dG and dU: a streaming pass (6 or 8 bytes read and 2 written per value). 16
// lanes hold a 1 x 128 block, 8 values each; both gradients are taken from one
// sigma, in pairs of fp32 operations, and their blocks' largest magnitudes meet by
// shuffles. 2048 x 11008 bf16: 30.9 us, 5.8 TB/s (with two blocks a half-warp in
// flight, 58 registers instead of 40, 0.5 us more).
template <int kElem>
struct Run {               // 8 values as they lie in memory
  uint4 v[kElem == kElemF32 ? 2 : 1];
};
template <int kElem>
__device__ __forceinline__ void load_run(Run<kElem>& r, const void* p, int64_t i) {
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const typename Elem<kElem>::T*>(p) + i);
  r.v[0] = __ldcs(q);
  if constexpr (kElem == kElemF32) r.v[1] = __ldcs(q + 1);
}
template <int kElem>
__device__ __forceinline__ void widen(const Run<kElem>& r, uint64_t (&v)[4]) {
  if constexpr (kElem == kElemF32) {
    v[0] = pair_of(__uint_as_float(r.v[0].x), __uint_as_float(r.v[0].y));
    v[1] = pair_of(__uint_as_float(r.v[0].z), __uint_as_float(r.v[0].w));
    v[2] = pair_of(__uint_as_float(r.v[1].x), __uint_as_float(r.v[1].y));
    v[3] = pair_of(__uint_as_float(r.v[1].z), __uint_as_float(r.v[1].w));
  } else {
    const uint32_t u[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack2<kElem>(u[j]);
      v[j] = pair_of(f.x, f.y);
    }
  }
}

// 8 values times `inverse` as e4m3 codes.
__device__ __forceinline__ uint2 codes_of(const uint64_t (&v)[4], float inverse) {
  const uint64_t i2 = pair_of(inverse, inverse);
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = both(mul2(v[j], i2));
    w[j] = e4m3x2(f.x, f.y);
  }
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

template <int kElem, bool kCubic>
__global__ void __launch_bounds__(256)
gated_bwd_kernel(const void* __restrict__ dy, const void* __restrict__ g, const void* __restrict__ u,
                 int64_t rows, int64_t cols, uint32_t nb, Curve c, uint8_t* __restrict__ dg,
                 float* __restrict__ dg_scale, uint8_t* __restrict__ du, float* __restrict__ du_scale) {
  let_next_start();
  wait_for_previous();
  const int64_t blocks = rows * nb, b = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  const int64_t r = blocks <= UINT32_MAX ? static_cast<uint32_t>(b) / nb : b / nb;
  const int64_t col = (b - r * nb) * kFp8Block + 8 * (threadIdx.x & 15), at = r * cols + col;
  const bool in = b < blocks && col < cols;
  Run<kElem> rd = {};
  Run<kElemBf16> rg = {}, ru = {};
  if (in) {
    load_run<kElem>(rd, dy, at);
    load_run<kElemBf16>(rg, g, at);
    load_run<kElemBf16>(ru, u, at);
  }
  uint64_t d[4], gv[4], uv[4];
  widen<kElem>(rd, d);
  widen<kElemBf16>(rg, gv);
  widen<kElemBf16>(ru, uv);
  float ag = 0.0f, au = 0.0f;
  const uint64_t one = pair_of(1.0f, 1.0f), minus = pair_of(-1.0f, -1.0f);
  const uint64_t k0 = pair_of(c.k0, c.k0), k1 = pair_of(c.k1, c.k1), c0 = pair_of(c.c0, c.c0);
  const uint64_t c13 = pair_of(3.0f * c.c1, 3.0f * c.c1);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint64_t g2 = 0;
    if (kCubic) {                       // p' stays finite where s (1 - s) is 0
      const float2 q = both(mul2(gv[j], gv[j]));
      g2 = pair_of(fminf(q.x, 1e30f), fminf(q.y, 1e30f));
    }
    const float2 t = both(mul2(gv[j], kCubic ? fma2(k1, g2, k0) : k0));
    const uint64_t s = pair_of(sigma_of(t.x), sigma_of(t.y)), f = mul2(gv[j], s);
    uint64_t slope = mul2(f, fma2(s, minus, one));
    slope = kCubic ? fma2(slope, fma2(c13, g2, c0), s) : add2(slope, s);
    uv[j] = mul2(mul2(d[j], uv[j]), slope);
    d[j] = mul2(d[j], f);
    const float2 x = both(uv[j]), y = both(d[j]);
    ag = max_abs(ag, x.x, x.y);
    au = max_abs(au, y.x, y.y);
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    ag = max_nan(ag, __shfl_xor_sync(0xffffffffu, ag, o));
    au = max_nan(au, __shfl_xor_sync(0xffffffffu, au, o));
  }
  const float sg = fp8_scale(ag), su = fp8_scale(au);
  if (in) {
    *reinterpret_cast<uint2*>(dg + at) = codes_of(uv, fp8_inverse(sg));
    *reinterpret_cast<uint2*>(du + at) = codes_of(d, fp8_inverse(su));
  }
  if ((threadIdx.x & 15) == 0 && b < blocks) {
    dg_scale[b] = sg;
    du_scale[b] = su;
  }
}

}  // namespace

cudaError_t launch_gated_bwd(const void* dy, int dy_elem, const void* g, const void* u, int64_t rows,
                             int64_t cols, Curve curve, uint8_t* dg, float* dg_scale, uint8_t* du,
                             float* du_scale, cudaStream_t st) {
  const int64_t nb = (cols + kFp8Block - 1) / kFp8Block;
  auto go = [&](auto elem) {
    constexpr int kElem = decltype(elem)::value;
    return launch_next(curve.k1 == 0.0f ? gated_bwd_kernel<kElem, false> : gated_bwd_kernel<kElem, true>,
                       (rows * nb + 15) / 16, 256, st, dy, g, u, rows, cols, nb, curve, dg,
                       dg_scale, du, du_scale);
  };
  if (dy_elem == kElemF32) return go(std::integral_constant<int, kElemF32>{});
  if (dy_elem == kElemBf16) return go(std::integral_constant<int, kElemBf16>{});
  return go(std::integral_constant<int, kElemF16>{});
}

}  // namespace nf4
