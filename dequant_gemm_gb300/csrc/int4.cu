// Uniform 4-bit weights in groups of 32, 64 or 128 along a row, each with a
// 16-bit scale and (optionally) a zero point: quantization, dequantization and
// products of few tokens. include/nf4gemm.h states the format.
#include "gated.cuh"

namespace nf4 {
namespace {

__device__ __forceinline__ float scale_value(uint32_t bits, bool bf16) {
  return bf16 ? __uint_as_float(bits << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}

// 8 consecutive values a thread, a group in kGroup / 8 neighbouring lanes.
template <int kElem, int kGroup, bool kZero>
__global__ void __launch_bounds__(256)
int4_quantize_kernel(const void* __restrict__ w, int64_t runs, bool bf16, uint32_t* __restrict__ codes,
                     uint16_t* __restrict__ scale, uint8_t* __restrict__ zero) {
  let_next_start();
  wait_for_previous();
  constexpr int kLanes = kGroup / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  float v[8] = {};
  if (i < runs) load8<kElem>(w, 8 * i, v);
  float lo = 0.0f, hi = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    lo = fminf(lo, kZero ? v[j] : -fabsf(v[j]));
    hi = fmaxf(hi, v[j]);
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    if (kZero) hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const float range = kZero ? __fdiv_rn(__fsub_rn(hi, lo), 15.0f) : __fdiv_rn(-lo, 7.0f);
  const uint32_t bits = bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(range))
                             : __half_as_ushort(__float2half_rn(range));
  const float s = scale_value(bits, bf16);
  float z = kZero ? 0.0f : 8.0f;
  if (kZero && s != 0.0f) z = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f);
  uint32_t out = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float q = s == 0.0f ? z : fminf(fmaxf(rintf(__fdiv_rn(v[j], s)) + z, 0.0f), 15.0f);
    out |= static_cast<uint32_t>(q) << (4 * (j ^ 1));     // the even element in the high half
  }
  if (i >= runs) return;
  codes[i] = out;
  if (i % kLanes == 0) {
    scale[i / kLanes] = static_cast<uint16_t>(bits);
    if (kZero) zero[i / kLanes] = static_cast<uint8_t>(z);
  }
}

template <int kElem>
__global__ void __launch_bounds__(256)
int4_dequantize_kernel(const uint32_t* __restrict__ codes, const uint16_t* __restrict__ scale,
                       const uint8_t* __restrict__ zero, int64_t runs, int lanes_log, bool bf16,
                       void* __restrict__ out) {
  let_next_start();
  wait_for_previous();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= runs) return;
  const uint32_t q = codes[i];
  const float s = scale_value(scale[i >> lanes_log], bf16);
  const int z = zero ? zero[i >> lanes_log] : 8;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = static_cast<float>(static_cast<int>((q >> (4 * (j ^ 1))) & 15) - z) * s;
  store8<kElem>(out, 8 * i, v);
}

// One warp an output.
__global__ void __launch_bounds__(256) int4_matmul_kernel(const Int4Call p) {
  const int64_t n = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5, m = blockIdx.y;
  const int lane = threadIdx.x & 31;
  if (n >= p.w[0].rows) return;
  float sum[2] = {};
  for (int mat = 0; mat < (p.gated ? 2 : 1); ++mat) {
    const nf4_int4_weight& w = p.w[mat];
    const bool bf16 = w.scale_elem == kElemBf16;
    for (int64_t k = lane; k < w.cols; k += 32) {
      const int64_t j = (n * w.cols + k) / w.group;
      const int q = (w.codes[(n * w.cols + k) / 2] >> (k % 2 ? 0 : 4)) & 15;
      const float v = static_cast<float>(q - (w.zero ? w.zero[j] : 8)) *
                      scale_value(static_cast<const uint16_t*>(w.scale)[j], bf16);
      const uint16_t x = static_cast<const uint16_t*>(p.x)[m * w.cols + k];
      sum[mat] = fmaf(v, scale_value(x, !p.x_f16), sum[mat]);
    }
    for (int o = 16; o > 0; o >>= 1) sum[mat] += __shfl_xor_sync(0xffffffffu, sum[mat], o);
  }
  if (lane != 0) return;
  float y = p.gated ? gated(sum[0], sum[1], p.curve) : sum[0];
  const int64_t at = m * p.w[0].rows + n;
  if (p.y_elem == kElemF32) {
    float* o = static_cast<float*>(p.y) + at;
    *o = y + (p.accumulate ? *o : 0.0f);
  } else if (p.y_elem == kElemBf16) {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.y) + at;
    *o = __float2bfloat16_rn(y + (p.accumulate ? __bfloat162float(*o) : 0.0f));
  } else {
    __half* o = static_cast<__half*>(p.y) + at;
    *o = __float2half_rn(y + (p.accumulate ? __half2float(*o) : 0.0f));
  }
}

template <typename F>
cudaError_t with_elem(int elem, F&& go) {
  if (elem == kElemF32) return go(std::integral_constant<int, kElemF32>{});
  if (elem == kElemBf16) return go(std::integral_constant<int, kElemBf16>{});
  return go(std::integral_constant<int, kElemF16>{});
}
template <typename F>
cudaError_t with_group(int group, F&& go) {
  if (group == 32) return go(std::integral_constant<int, 32>{});
  if (group == 64) return go(std::integral_constant<int, 64>{});
  return go(std::integral_constant<int, 128>{});
}

}  // namespace

cudaError_t launch_int4_quantize(const void* w, int w_elem, int64_t rows, int64_t cols, int group,
                                 bool scale_bf16, uint8_t* codes, void* scale, uint8_t* zero,
                                 cudaStream_t st) {
  const int64_t runs = rows * cols / 8;
  return with_elem(w_elem, [&](auto elem) {
    return with_group(group, [&](auto g) {
      return launch_next(zero ? int4_quantize_kernel<decltype(elem)::value, decltype(g)::value, true>
                              : int4_quantize_kernel<decltype(elem)::value, decltype(g)::value, false>,
                         (runs + 255) / 256, 256, st, w, runs, scale_bf16,
                         reinterpret_cast<uint32_t*>(codes), static_cast<uint16_t*>(scale), zero);
    });
  });
}

cudaError_t launch_int4_dequantize(const nf4_int4_weight& w, void* out, int out_elem, cudaStream_t st) {
  const int64_t runs = w.rows * w.cols / 8;
  return with_elem(out_elem, [&](auto elem) {
    return launch_next(int4_dequantize_kernel<decltype(elem)::value>, (runs + 255) / 256, 256, st,
                       reinterpret_cast<const uint32_t*>(w.codes), static_cast<const uint16_t*>(w.scale), w.zero,
                       runs, w.group == 32 ? 2 : w.group == 64 ? 3 : 4, w.scale_elem == kElemBf16, out);
  });
}

cudaError_t launch_int4_matmul(const Int4Call& c) {
  const int64_t grid = (c.w[0].rows + 7) / 8;
  int4_matmul_kernel<<<dim3(static_cast<unsigned>(grid), static_cast<unsigned>(c.M)), 256, 0, c.st>>>(c);
  return cudaGetLastError();
}

}  // namespace nf4
