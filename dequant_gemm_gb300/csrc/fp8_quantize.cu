// Block-scaled e4m3 quantization of activations and gradients (one fp32 scale
// for each 1 x 128 block) and of weights (128 x 128), and the stand-alone
// dequantization. The format is stated in fp8.cuh.
//
// All kernels are streaming passes: 4 or 2 bytes read and 1 byte and a
// little written per value (dequantize the reverse). Measured, of the copy
// bandwidth: 1 x 128 blocks of 4096 x 18944 bf16 39 us (0.89), 128 x 128 blocks
// of 11008 x 4096 fp32 34 us (0.99).
#include "fp8.cuh"

namespace nf4 {
namespace {

// 1 x 128 blocks: 16 lanes hold a block, 8 values each, so a half-warp's load
// is a whole 256-byte (16-bit input) or 512-byte (fp32) run and its store a
// whole 128-byte line of codes. kRowUnroll blocks per half-warp keep that many
// loads in flight per lane.
constexpr int kRowThreads = 256;
constexpr int kRowUnroll = 4;

// kWhole: rows of whole blocks, which then lie one after another and need no
// row index (with a 64-bit division by kb for each block the pass above took
// 74 us).
template <int kElem, bool kWhole>
__global__ void __launch_bounds__(kRowThreads)
fp8_quantize_rows_kernel(const void* __restrict__ x, int64_t rows, int64_t cols, uint32_t kb,
                         uint8_t* __restrict__ codes, float* __restrict__ scale) {
  let_next_start();
  wait_for_previous();
  const int sub = threadIdx.x & 15;
  const int64_t groups = rows * kb;
  const int64_t g0 = (static_cast<int64_t>(blockIdx.x) * (kRowThreads / 16) + (threadIdx.x >> 4)) * kRowUnroll;
  float v[kRowUnroll][8];
  int64_t at[kRowUnroll];
#pragma unroll
  for (int u = 0; u < kRowUnroll; ++u) {
    const int64_t g = g0 + u;
    if (kWhole) {
      at[u] = g < groups ? g * kFp8Block + 8 * sub : -1;
    } else {
      const int64_t r = groups <= UINT32_MAX ? static_cast<uint32_t>(g) / kb : g / kb;
      const int64_t c = (g - r * kb) * kFp8Block + 8 * sub;
      at[u] = g < groups && c < cols ? r * cols + c : -1;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[u][j] = 0.0f;
    if (at[u] >= 0) load8<kElem>(x, at[u], v[u]);
  }
#pragma unroll
  for (int u = 0; u < kRowUnroll; ++u) {
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) a = max_nan(a, fabsf(v[u][j]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
    const float s = fp8_scale(a), inv = fp8_inverse(s);
    if (at[u] >= 0)
      *reinterpret_cast<uint2*>(codes + at[u]) =
          make_uint2(e4m3x4(v[u][0] * inv, v[u][1] * inv, v[u][2] * inv, v[u][3] * inv),
                     e4m3x4(v[u][4] * inv, v[u][5] * inv, v[u][6] * inv, v[u][7] * inv));
    if (sub == 0 && g0 + u < groups) scale[g0 + u] = s;
  }
}

// 128 x 128 blocks: one CTA a block, held in registers between the maximum
// and the rounding.
constexpr int kTileThreads = 256;

template <int kElem>
__global__ void __launch_bounds__(kTileThreads)
fp8_quantize_tiles_kernel(const void* __restrict__ x, int64_t rows, int64_t cols, int kb,
                          uint8_t* __restrict__ codes, float* __restrict__ scale) {
  constexpr int kSteps = kFp8Block * kFp8Block / (8 * kTileThreads);   // 8
  __shared__ float part[kTileThreads / 32];
  let_next_start();
  wait_for_previous();
  const int64_t rb = blockIdx.x / kb, cb = blockIdx.x % kb;
  const int64_t c = cb * kFp8Block + 8 * (threadIdx.x & 15);
  const int64_t r0 = rb * kFp8Block + (threadIdx.x >> 4);
  float v[kSteps][8];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t r = r0 + i * (kTileThreads / 16);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    if (r < rows && c < cols) load8<kElem>(x, r * cols + c, v[i]);
  }
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < kSteps; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) a = max_nan(a, fabsf(v[i][j]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kTileThreads / 32; ++i) a = max_nan(a, part[i]);
  const float s = fp8_scale(a), inv = fp8_inverse(s);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t r = r0 + i * (kTileThreads / 16);
    if (r < rows && c < cols)
      *reinterpret_cast<uint2*>(codes + r * cols + c) =
          make_uint2(e4m3x4(v[i][0] * inv, v[i][1] * inv, v[i][2] * inv, v[i][3] * inv),
                     e4m3x4(v[i][4] * inv, v[i][5] * inv, v[i][6] * inv, v[i][7] * inv));
  }
  if (threadIdx.x == 0) scale[blockIdx.x] = s;
}

// One thread per 8 values.
template <int kElem>
__global__ void __launch_bounds__(256)
fp8_dequantize_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scale,
                      int64_t cols, int64_t chunks, int kb, int block_rows, void* __restrict__ out) {
  let_next_start();
  wait_for_previous();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (t >= chunks) return;
  const int64_t i = 8 * t, r = i / cols, c = i - r * cols;
  const uint2 q = *reinterpret_cast<const uint2*>(codes + i);
  const float s = scale[(r / block_rows) * kb + c / kFp8Block];
  float v[8];
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = e4m3x2_to_float2(static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1))));
    v[2 * j] = f.x * s;
    v[2 * j + 1] = f.y * s;
  }
  store8<kElem>(out, i, v);
}

}  // namespace

cudaError_t launch_fp8_quantize(const void* x, int x_elem, int64_t rows, int64_t cols,
                                int block_rows, uint8_t* codes, float* scale, cudaStream_t st) {
  const int64_t kb = (cols + kFp8Block - 1) / kFp8Block;
  auto go = [&](auto elem) {
    constexpr int kElem = decltype(elem)::value;
    if (block_rows == 1) {
      const int64_t per_cta = kRowThreads / 16 * kRowUnroll;
      return launch_next(cols % kFp8Block == 0 ? fp8_quantize_rows_kernel<kElem, true>
                                               : fp8_quantize_rows_kernel<kElem, false>,
                         (rows * kb + per_cta - 1) / per_cta, kRowThreads, st, x, rows, cols, kb, codes,
                         scale);
    }
    return launch_next(fp8_quantize_tiles_kernel<kElem>, (rows + kFp8Block - 1) / kFp8Block * kb,
                       kTileThreads, st, x, rows, cols, kb, codes, scale);
  };
  if (x_elem == kElemF32) return go(std::integral_constant<int, kElemF32>{});
  if (x_elem == kElemBf16) return go(std::integral_constant<int, kElemBf16>{});
  return go(std::integral_constant<int, kElemF16>{});
}

cudaError_t launch_fp8_dequantize(const uint8_t* codes, const float* scale, int64_t rows,
                                  int64_t cols, int block_rows, void* out, int out_elem,
                                  cudaStream_t st) {
  const int64_t kb = (cols + kFp8Block - 1) / kFp8Block, chunks = rows * cols / 8;
  auto go = [&](auto elem) {
    constexpr int kElem = decltype(elem)::value;
    return launch_next(fp8_dequantize_kernel<kElem>, (chunks + 255) / 256, 256, st, codes, scale, cols,
                       chunks, kb, block_rows, out);
  };
  if (out_elem == kElemF32) return go(std::integral_constant<int, kElemF32>{});
  if (out_elem == kElemBf16) return go(std::integral_constant<int, kElemBf16>{});
  return go(std::integral_constant<int, kElemF16>{});
}

}  // namespace nf4
