// The gradients of the gated block's product (gated.cuh), in 8 bits for the two
// products that make the input gradient of them (fp8_gemm.cu):
//   dG = dY U act'(G), dU = dY act(G),
//   act'(g) = s + g s (1 - s) p'(g), s = sigma(p(g)), p'(g) = c0 + 3 c1 g^2
#include "gated.cuh"

namespace nf4 {
namespace {

// dG and dU: a streaming pass (6 or 8 bytes read and 2 written per value). 16
// lanes hold a 1 x 128 block, 8 values each; both gradients are taken from one
// sigma, and their blocks' largest magnitudes meet by shuffles. kUnroll blocks a
// half-warp keep that many of each load in flight.
constexpr int kUnroll = 2;

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
__device__ __forceinline__ void widen(const Run<kElem>& r, float (&v)[8]) {
  if constexpr (kElem == kElemF32) {
    v[0] = __uint_as_float(r.v[0].x); v[1] = __uint_as_float(r.v[0].y);
    v[2] = __uint_as_float(r.v[0].z); v[3] = __uint_as_float(r.v[0].w);
    v[4] = __uint_as_float(r.v[1].x); v[5] = __uint_as_float(r.v[1].y);
    v[6] = __uint_as_float(r.v[1].z); v[7] = __uint_as_float(r.v[1].w);
  } else {
    const uint32_t u[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack2<kElem>(u[j]);
      v[2 * j] = f.x;
      v[2 * j + 1] = f.y;
    }
  }
}

template <int kElem, bool kCubic>
__global__ void __launch_bounds__(256)
gated_bwd_kernel(const void* __restrict__ dy, const void* __restrict__ g, const void* __restrict__ u,
                 int64_t rows, int64_t cols, uint32_t nb, Curve c, uint8_t* __restrict__ dg,
                 float* __restrict__ dg_scale, uint8_t* __restrict__ du, float* __restrict__ du_scale) {
  let_next_start();
  wait_for_previous();
  const int64_t blocks = rows * nb, b0 = (static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4)) * kUnroll;
  Run<kElem> rd[kUnroll] = {};
  Run<kElemBf16> rg[kUnroll] = {}, ru[kUnroll] = {};
  int64_t at[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int64_t b = b0 + i;
    const int64_t r = blocks <= UINT32_MAX ? static_cast<uint32_t>(b) / nb : b / nb;
    const int64_t col = (b - r * nb) * kFp8Block + 8 * (threadIdx.x & 15);
    at[i] = b < blocks && col < cols ? r * cols + col : -1;
    if (at[i] < 0) continue;
    load_run<kElem>(rd[i], dy, at[i]);
    load_run<kElemBf16>(rg[i], g, at[i]);
    load_run<kElemBf16>(ru[i], u, at[i]);
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    float d[8], gv[8], uv[8];
    widen<kElem>(rd[i], d);
    widen<kElemBf16>(rg[i], gv);
    widen<kElemBf16>(ru[i], uv);
    float ag = 0.0f, au = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float g2 = kCubic ? fminf(gv[j] * gv[j], 1e30f) : 0.0f;    // p' stays finite where s (1 - s) is 0
      const float s = sigma_of(gv[j] * (kCubic ? fmaf(c.k1, g2, c.k0) : c.k0)), f = gv[j] * s;
      const float slope = fmaf(f * (1.0f - s), kCubic ? fmaf(3.0f * c.c1, g2, c.c0) : 1.0f, s);
      uv[j] = d[j] * uv[j] * slope;
      d[j] *= f;
      ag = max_nan(ag, fabsf(uv[j]));
      au = max_nan(au, fabsf(d[j]));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      ag = max_nan(ag, __shfl_xor_sync(0xffffffffu, ag, o));
      au = max_nan(au, __shfl_xor_sync(0xffffffffu, au, o));
    }
    const float sg = fp8_scale(ag), su = fp8_scale(au), ig = fp8_inverse(sg), iu = fp8_inverse(su);
    if (at[i] >= 0) {
      *reinterpret_cast<uint2*>(dg + at[i]) =
          make_uint2(e4m3x4(uv[0] * ig, uv[1] * ig, uv[2] * ig, uv[3] * ig),
                     e4m3x4(uv[4] * ig, uv[5] * ig, uv[6] * ig, uv[7] * ig));
      *reinterpret_cast<uint2*>(du + at[i]) = make_uint2(e4m3x4(d[0] * iu, d[1] * iu, d[2] * iu, d[3] * iu),
                                                         e4m3x4(d[4] * iu, d[5] * iu, d[6] * iu, d[7] * iu));
    }
    if ((threadIdx.x & 15) == 0 && b0 + i < blocks) {
      dg_scale[b0 + i] = sg;
      du_scale[b0 + i] = su;
    }
  }
}

}  // namespace

cudaError_t launch_gated_bwd(const void* dy, int dy_elem, const void* g, const void* u, int64_t rows,
                             int64_t cols, Curve curve, uint8_t* dg, float* dg_scale, uint8_t* du,
                             float* du_scale, cudaStream_t st) {
  const int64_t nb = (cols + kFp8Block - 1) / kFp8Block;
  const int64_t per_cta = 16 * kUnroll;
  auto go = [&](auto elem) {
    constexpr int kElem = decltype(elem)::value;
    return launch_next(curve.k1 == 0.0f ? gated_bwd_kernel<kElem, false> : gated_bwd_kernel<kElem, true>,
                       (rows * nb + per_cta - 1) / per_cta, 256, st, dy, g, u, rows, cols, nb, curve, dg,
                       dg_scale, du, du_scale);
  };
  if (dy_elem == kElemF32) return go(std::integral_constant<int, kElemF32>{});
  if (dy_elem == kElemBf16) return go(std::integral_constant<int, kElemBf16>{});
  return go(std::integral_constant<int, kElemF16>{});
}

}  // namespace nf4
