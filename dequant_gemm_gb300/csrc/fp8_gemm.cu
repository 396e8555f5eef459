// Products of block-scaled e4m3 operands (fp8.cuh):
//   forward    Y[m, n]  = sum_b sx[m, b] sw[n / 128, b] sum_{k in b} qx[m, k] qw[n, k]
//   input grad dX[m, k] = sum_b sy[m, b] sw[b, k / 128] sum_{n in b} qy[m, n] qw[n, k]
// (b: the 128-wide blocks of the reduction; the weight is frozen, so there is
// no weight gradient.)
#include <algorithm>

#include "fp8.cuh"

namespace nf4 {
namespace {

struct MatmulArgs {
  const uint8_t *a, *w;
  const float *a_scale, *w_scale;
  int64_t M, red, cols;    // out [M, cols]
  int64_t w_pitch;         // K
  int rb, kb;              // blocks along the reduction and along K
  void* out;
  int out_bf16, accumulate;
};

// 64 x 64 outputs a CTA, 4 x 4 a thread, one 128-wide block at a time staged
// in shared memory as fp32 in two halves of 64.
template <bool kDx>
__global__ void __launch_bounds__(256) fp8_matmul_simple_kernel(const MatmulArgs p) {
  __shared__ float As[64][65], Bs[64][65];   // [reduction][token], [reduction][column]
  const int64_t m0 = blockIdx.y * 64ll, c0 = blockIdx.x * 64ll;
  const int tm = (threadIdx.x >> 4) * 4, tc = (threadIdx.x & 15) * 4;
  float acc[4][4] = {};
  for (int b = 0; b < p.rb; ++b) {
    float t[4][4] = {};
    for (int half = 0; half < 2; ++half) {
      const int64_t r0 = b * 128ll + half * 64;
      __syncthreads();
      for (int e = threadIdx.x; e < 64 * 32; e += 256) {
        const int i = e >> 5, r = (e & 31) * 2;
        float2 v = make_float2(0.f, 0.f);
        if (m0 + i < p.M && r0 + r < p.red)
          v = e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(p.a + (m0 + i) * p.red + r0 + r));
        As[r][i] = v.x;
        As[r + 1][i] = v.y;
        float2 u = make_float2(0.f, 0.f);
        if constexpr (kDx) {   // weight row r0 + i, columns c0 + r, + 1
          if (r0 + i < p.red && c0 + r < p.cols)
            u = e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(p.w + (r0 + i) * p.w_pitch + c0 + r));
          Bs[i][r] = u.x;
          Bs[i][r + 1] = u.y;
        } else {
          if (c0 + i < p.cols && r0 + r < p.red)
            u = e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(p.w + (c0 + i) * p.w_pitch + r0 + r));
          Bs[r][i] = u.x;
          Bs[r + 1][i] = u.y;
        }
      }
      __syncthreads();
      for (int r = 0; r < 64; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) t[i][j] += As[r][tm + i] * Bs[r][tc + j];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + tm + i, c = c0 + tc + j;
        if (m < p.M && c < p.cols) {
          const float sw = kDx ? p.w_scale[static_cast<int64_t>(b) * p.kb + c / 128]
                               : p.w_scale[c / 128 * p.kb + b];
          acc[i][j] += p.a_scale[m * p.rb + b] * sw * t[i][j];
        }
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + tm + i, c = c0 + tc + j;
      if (m >= p.M || c >= p.cols) continue;
      float v = acc[i][j];
      if (p.out_bf16) {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + m * p.cols + c;
        if (p.accumulate) v += __bfloat162float(*o);
        *o = __float2bfloat16_rn(v);
      } else {
        float* o = static_cast<float*>(p.out) + m * p.cols + c;
        if (p.accumulate) v += *o;
        *o = v;
      }
    }
}

}  // namespace

cudaError_t launch_fp8_matmul(const Fp8Call& c) {
  MatmulArgs a;
  a.a = c.a;
  a.w = c.w;
  a.a_scale = c.a_scale;
  a.w_scale = c.w_scale;
  a.M = c.M;
  a.red = c.dx ? c.N : c.K;
  a.cols = c.dx ? c.K : c.N;
  a.w_pitch = c.K;
  a.rb = static_cast<int>((a.red + 127) / 128);
  a.kb = static_cast<int>((c.K + 127) / 128);
  a.out = c.out;
  a.out_bf16 = c.out_bf16;
  a.accumulate = c.accumulate;
  const dim3 grid(static_cast<unsigned>((a.cols + 63) / 64), static_cast<unsigned>((a.M + 63) / 64));
  if (c.dx) fp8_matmul_simple_kernel<true><<<grid, 256, 0, c.st>>>(a);
  else fp8_matmul_simple_kernel<false><<<grid, 256, 0, c.st>>>(a);
  return cudaGetLastError();
}

}  // namespace nf4
