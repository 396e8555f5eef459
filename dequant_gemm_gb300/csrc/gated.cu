// The gated feed-forward block on block-scaled e4m3 operands (fp8.cuh):
//   forward   G = X Wg^T, U = X Wu^T, Y = act(G) * U
//   backward  dG = dY U act'(G), dU = dY act(G), dX = dG Wg + dU Wu
#include "gated.cuh"

namespace nf4 {
namespace {

constexpr int kTok = 8;       // tokens a CTA
constexpr int kPitch = 132;   // floats of a staged weight row, off the banks' period

__device__ float code_value(uint8_t q) { return e4m3x2_to_float2(q).x; }

// One thread an output column, kTok tokens; a 128 x 128 block of a weight at a
// time in shared memory, widened.
__global__ void __launch_bounds__(128)
gated_fwd_kernel(const GatedFwdCall p, int kb, int nb) {
  extern __shared__ float sm[];
  float* w = sm;
  float* x = sm + 128 * kPitch;
  __shared__ float part[4];
  const int col = threadIdx.x;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 128, m0 = static_cast<int64_t>(blockIdx.y) * kTok;
  float sum[2][kTok] = {};
  for (int b = 0; b < kb; ++b) {
    const int64_t k0 = static_cast<int64_t>(b) * 128;
    for (int mat = 0; mat < 2; ++mat) {
      const uint8_t* codes = mat ? p.wu : p.wg;
      __syncthreads();
      for (int i = threadIdx.x; i < 128 * 128; i += 128) {
        const int64_t r = n0 + i / 128, k = k0 + i % 128;
        w[i / 128 * kPitch + i % 128] = r < p.N && k < p.K ? code_value(codes[r * p.K + k]) : 0.0f;
      }
      for (int i = threadIdx.x; i < kTok * 128; i += 128) {
        const int64_t r = m0 + i / 128, k = k0 + i % 128;
        x[i] = r < p.M && k < p.K ? code_value(p.a[r * p.K + k]) : 0.0f;
      }
      __syncthreads();
      const float sw = (mat ? p.wu_scale : p.wg_scale)[n0 / 128 * kb + b];
      for (int t = 0; t < kTok && m0 + t < p.M; ++t) {
        float s = 0.0f;
        for (int k = 0; k < 128; ++k) s = fmaf(x[t * 128 + k], w[col * kPitch + k], s);
        sum[mat][t] = fmaf(s, p.a_scale[(m0 + t) * kb + b] * sw, sum[mat][t]);
      }
    }
  }
  for (int t = 0; t < kTok && m0 + t < p.M; ++t) {
    const bool in = n0 + col < p.N;
    const float g = sum[0][t], u = sum[1][t], y = gated(g, u, p.curve);
    const int64_t at = (m0 + t) * p.N + n0 + col;
    if (in && p.g) {
      static_cast<__nv_bfloat16*>(p.g)[at] = __float2bfloat16_rn(g);
      static_cast<__nv_bfloat16*>(p.u)[at] = __float2bfloat16_rn(u);
    }
    if (p.y_fp8) {
      float a = in ? fabsf(y) : 0.0f;
      for (int o = 16; o > 0; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
      __syncthreads();
      if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = a;
      __syncthreads();
      const float s = fp8_scale(max_nan(max_nan(part[0], part[1]), max_nan(part[2], part[3])));
      if (in) static_cast<uint8_t*>(p.y)[at] = static_cast<uint8_t>(e4m3x2(y * fp8_inverse(s), 0.0f));
      if (threadIdx.x == 0) p.scale[(m0 + t) * nb + n0 / 128] = s;
    } else if (in && p.y_bf16) {
      static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(y);
    } else if (in) {
      static_cast<float*>(p.y)[at] = y;
    }
  }
}

__global__ void __launch_bounds__(128) gated_dx_kernel(const GatedDxCall p, int kb, int nb) {
  extern __shared__ float sm[];
  float* w = sm;
  float* x = sm + 128 * kPitch;
  const int col = threadIdx.x;
  const int64_t k0 = static_cast<int64_t>(blockIdx.x) * 128, m0 = static_cast<int64_t>(blockIdx.y) * kTok;
  float sum[kTok] = {};
  for (int i = 0; i < 2 * nb; ++i) {
    const bool up = i >= nb;
    const int b = up ? i - nb : i;
    const int64_t n0 = static_cast<int64_t>(b) * 128;
    const uint8_t* codes = up ? p.wu : p.wg;
    const uint8_t* d = up ? p.du : p.dg;
    __syncthreads();
    for (int j = threadIdx.x; j < 128 * 128; j += 128) {
      const int64_t r = n0 + j / 128, k = k0 + j % 128;
      w[j / 128 * kPitch + j % 128] = r < p.N && k < p.K ? code_value(codes[r * p.K + k]) : 0.0f;
    }
    for (int j = threadIdx.x; j < kTok * 128; j += 128) {
      const int64_t r = m0 + j / 128, n = n0 + j % 128;
      x[j] = r < p.M && n < p.N ? code_value(d[r * p.N + n]) : 0.0f;
    }
    __syncthreads();
    const float sw = (up ? p.wu_scale : p.wg_scale)[b * static_cast<int64_t>(kb) + blockIdx.x];
    for (int t = 0; t < kTok && m0 + t < p.M; ++t) {
      float s = 0.0f;
      for (int n = 0; n < 128; ++n) s = fmaf(x[t * 128 + n], w[n * kPitch + col], s);
      sum[t] = fmaf(s, (up ? p.du_scale : p.dg_scale)[(m0 + t) * nb + b] * sw, sum[t]);
    }
  }
  for (int t = 0; t < kTok && m0 + t < p.M && k0 + col < p.K; ++t) {
    const int64_t at = (m0 + t) * p.K + k0 + col;
    if (p.out_bf16) {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + at;
      *o = __float2bfloat16_rn(sum[t] + (p.accumulate ? __bfloat162float(*o) : 0.0f));
    } else {
      float* o = static_cast<float*>(p.out) + at;
      *o = sum[t] + (p.accumulate ? *o : 0.0f);
    }
  }
}

constexpr int kSimpleSmem = (128 * kPitch + kTok * 128) * 4;

// dG and dU: a streaming pass (6 or 8 bytes read and 2 written per value). 16
// lanes hold a 1 x 128 block, 8 values each; both gradients are taken from one
// sigma, and their blocks' largest magnitudes meet by shuffles.
template <int kElem>
__global__ void __launch_bounds__(256)
gated_bwd_kernel(const void* __restrict__ dy, const void* __restrict__ g, const void* __restrict__ u,
                 int64_t rows, int64_t cols, uint32_t nb, Curve c, uint8_t* __restrict__ dg,
                 float* __restrict__ dg_scale, uint8_t* __restrict__ du, float* __restrict__ du_scale) {
  let_next_start();
  wait_for_previous();
  const int64_t blocks = rows * nb, b = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  const int64_t r = blocks <= UINT32_MAX ? static_cast<uint32_t>(b) / nb : b / nb;
  const int64_t col = (b - r * nb) * kFp8Block + 8 * (threadIdx.x & 15);
  const bool in = b < blocks && col < cols;
  const int64_t at = r * cols + col;
  float d[8] = {}, gv[8] = {}, uv[8] = {};
  if (in) {
    load8<kElem>(dy, at, d);
    load8<kElemBf16>(g, at, gv);
    load8<kElemBf16>(u, at, uv);
  }
  float ag = 0.0f, au = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float s = gate_sigma(gv[j], c), f = gv[j] * s;
    const float slope = fmaf(f * (1.0f - s), fmaf(3.0f * c.c1, fminf(gv[j] * gv[j], 1e30f), c.c0), s);
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
  if (in) {
    *reinterpret_cast<uint2*>(dg + at) =
        make_uint2(e4m3x4(uv[0] * ig, uv[1] * ig, uv[2] * ig, uv[3] * ig),
                   e4m3x4(uv[4] * ig, uv[5] * ig, uv[6] * ig, uv[7] * ig));
    *reinterpret_cast<uint2*>(du + at) = make_uint2(e4m3x4(d[0] * iu, d[1] * iu, d[2] * iu, d[3] * iu),
                                                    e4m3x4(d[4] * iu, d[5] * iu, d[6] * iu, d[7] * iu));
  }
  if ((threadIdx.x & 15) == 0 && b < blocks) {
    dg_scale[b] = sg;
    du_scale[b] = su;
  }
}

}  // namespace

cudaError_t launch_gated_fwd(const GatedFwdCall& c) {
  const int kb = static_cast<int>((c.K + 127) / 128), nb = static_cast<int>((c.N + 127) / 128);
  static std::once_flag once[kOnceDevices];
  once_per_device(once, c.device, [] {
    cudaFuncSetAttribute(gated_fwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSimpleSmem);
  });
  gated_fwd_kernel<<<dim3(nb, static_cast<unsigned>((c.M + kTok - 1) / kTok)), 128, kSimpleSmem, c.st>>>(c, kb, nb);
  return cudaGetLastError();
}

cudaError_t launch_gated_dx(const GatedDxCall& c) {
  const int kb = static_cast<int>((c.K + 127) / 128), nb = static_cast<int>((c.N + 127) / 128);
  static std::once_flag once[kOnceDevices];
  once_per_device(once, c.device, [] {
    cudaFuncSetAttribute(gated_dx_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSimpleSmem);
  });
  gated_dx_kernel<<<dim3(kb, static_cast<unsigned>((c.M + kTok - 1) / kTok)), 128, kSimpleSmem, c.st>>>(c, kb, nb);
  return cudaGetLastError();
}

cudaError_t launch_gated_bwd(const void* dy, int dy_elem, const void* g, const void* u, int64_t rows,
                             int64_t cols, Curve curve, uint8_t* dg, float* dg_scale, uint8_t* du,
                             float* du_scale, cudaStream_t st) {
  const int64_t nb = (cols + kFp8Block - 1) / kFp8Block;
  auto go = [&](auto elem) {
    return launch_next(gated_bwd_kernel<decltype(elem)::value>, (rows * nb + 15) / 16, 256, st, dy, g, u,
                       rows, cols, nb, curve, dg, dg_scale, du, du_scale);
  };
  if (dy_elem == kElemF32) return go(std::integral_constant<int, kElemF32>{});
  if (dy_elem == kElemBf16) return go(std::integral_constant<int, kElemBf16>{});
  return go(std::integral_constant<int, kElemF16>{});
}

}  // namespace nf4
