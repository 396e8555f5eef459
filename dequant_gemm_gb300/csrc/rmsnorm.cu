// RMS norm with the residual's addition, forward and backward.
//
// Forward, per row:  h = rnd(x + r)  (rnd to the residual's type; without a
// residual h = x),  rstd = (mean(h^2) + eps)^(-1/2),  y = h rstd w.  y leaves
// as 16- or 32-bit values, or as block-scaled e4m3 (fp8.cuh) for the 8-bit
// products: the row is then read once and its codes and scales written
// directly, where a separate quantizer would write and read y again.
//
// Backward, with xh = h rstd and g = dy w:
//   dx = rstd (g - xh mean(g xh)) + dh      dw = sum over rows of dy xh
// dh is the gradient that reaches h from the residual stream, dx the gradient
// of both x and r. The row sums of dw are kept per CTA in fp32 and added in
// a fixed order by a second kernel, so results are repeatable.
//
// Sums and statistics are fp32; each output is rounded once.
#include <algorithm>

#include "fp8.cuh"

namespace nf4 {
namespace {

// kVec consecutive elements of runtime type `elem` at element i.
template <int kVec>
__device__ __forceinline__ void load_any(const void* p, int elem, int64_t i, float (&v)[kVec]) {
  if constexpr (kVec == 8) {
    if (elem == kElemF32) load8<kElemF32>(p, i, v);
    else if (elem == kElemBf16) load8<kElemBf16>(p, i, v);
    else load8<kElemF16>(p, i, v);
  } else {
    if (elem == kElemF32) v[0] = static_cast<const float*>(p)[i];
    else if (elem == kElemBf16) v[0] = __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    else v[0] = __half2float(static_cast<const __half*>(p)[i]);
  }
}

template <int kVec>
__device__ __forceinline__ void store_any(void* p, int elem, int64_t i, const float (&v)[kVec]) {
  if constexpr (kVec == 8) {
    if (elem == kElemF32) store8<kElemF32>(p, i, v);
    else if (elem == kElemBf16) store8<kElemBf16>(p, i, v);
    else store8<kElemF16>(p, i, v);
  } else {
    if (elem == kElemF32) static_cast<float*>(p)[i] = v[0];
    else if (elem == kElemBf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v[0]);
    else static_cast<__half*>(p)[i] = __float2half_rn(v[0]);
  }
}

// v rounded to the type `elem` and widened again.
__device__ __forceinline__ float round_to(float v, int elem) {
  if (elem == kElemBf16) return __bfloat162float(__float2bfloat16_rn(v));
  if (elem == kElemF16) return __half2float(__float2half_rn(v));
  return v;
}

// Sum over the CTA's threads, the same in every thread. part: 32 floats of
// shared memory; a second call needs a __syncthreads in between.
__device__ __forceinline__ float block_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  v = lane < warps ? part[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct FwdArgs {
  const void *x, *residual, *weight;
  void *h, *y;
  float *scale, *rstd;
  int64_t cols;
  int x_elem, h_elem, w_elem, y_elem, y_fp8;
  float eps;
};

// h of one run of kVec elements.
template <int kVec>
__device__ __forceinline__ void load_h(const FwdArgs& p, int64_t i, float (&v)[kVec]) {
  load_any<kVec>(p.x, p.x_elem, i, v);
  if (p.residual) {
    float r[kVec];
    load_any<kVec>(p.residual, p.h_elem, i, r);
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = round_to(v[j] + r[j], p.h_elem);
  }
}

// y of one run: rounded to its type, or to e4m3 codes, a block's 16 runs of 8
// being held by the 16 lanes of a half-warp (every lane takes part; runs past
// the row's end hold zeros).
template <int kVec>
__device__ __forceinline__ void write_y(const FwdArgs& p, int64_t row, int64_t c, bool in,
                                        const float (&y)[kVec]) {
  const int64_t i = row * p.cols + c;
  if constexpr (kVec == 8) {
    if (p.y_fp8) {
      float a = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) a = max_nan(a, fabsf(y[j]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
      const float s = fp8_scale(a), inv = fp8_inverse(s);
      if (in) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + i) =
            make_uint2(e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                       e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
        if ((threadIdx.x & 15) == 0)
          p.scale[row * ((p.cols + kFp8Block - 1) / kFp8Block) + c / kFp8Block] = s;
      }
      return;
    }
  }
  if (in) store_any<kVec>(p.y, p.y_elem, i, y);
}

// One CTA a row of any length, read twice: the second time h comes from where
// the first pass wrote it (each thread reads back its own elements).
template <int kVec>
__global__ void __launch_bounds__(512) rmsnorm_fwd_long_kernel(const FwdArgs p) {
  __shared__ float part[32];
  const int64_t row = blockIdx.x, step = static_cast<int64_t>(blockDim.x) * kVec;
  float ss = 0.0f;
  for (int64_t c = threadIdx.x * kVec; c < p.cols; c += step) {
    float v[kVec];
    load_h<kVec>(p, row * p.cols + c, v);
    if (p.residual) store_any<kVec>(p.h, p.h_elem, row * p.cols + c, v);
#pragma unroll
    for (int j = 0; j < kVec; ++j) ss += v[j] * v[j];
  }
  const float rstd = rsqrtf(block_sum(ss, part) / static_cast<float>(p.cols) + p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
  const void* src = p.residual ? p.h : p.x;
  const int elem = p.residual ? p.h_elem : p.x_elem;
  // whole half-warps stay together: a block's lanes all reach its maximum
  for (int64_t c0 = 0; c0 < p.cols; c0 += step) {
    const int64_t c = c0 + threadIdx.x * kVec;
    const bool in = c < p.cols;
    float y[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) y[j] = 0.0f;
    if (in) {
      float w[kVec];
      load_any<kVec>(src, elem, row * p.cols + c, y);
      load_any<kVec>(p.weight, p.w_elem, c, w);
#pragma unroll
      for (int j = 0; j < kVec; ++j) y[j] = y[j] * rstd * w[j];
    }
    write_y<kVec>(p, row, c, in, y);
  }
}

struct BwdArgs {
  const void *dy, *h, *dh, *weight;
  const float* rstd;
  void* dx;
  float* partial;
  int64_t rows, cols;
  int elem, w_elem;
};

// Rows of any length, gridDim.x CTAs taking them in turn: one pass for
// mean(g xh), a second for dx. The CTA's share of dw accumulates in its row of
// `partial` (each thread its own columns).
template <int kVec>
__global__ void __launch_bounds__(512) rmsnorm_bwd_long_kernel(const BwdArgs p) {
  __shared__ float part[2][32];
  const int64_t step = static_cast<int64_t>(blockDim.x) * kVec;
  float* acc = p.partial + blockIdx.x * p.cols;
  int k = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, ++k) {
    const float r = p.rstd[row];
    float dot = 0.0f;
    for (int64_t c = threadIdx.x * kVec; c < p.cols; c += step) {
      float g[kVec], h[kVec], w[kVec];
      load_any<kVec>(p.dy, p.elem, row * p.cols + c, g);
      load_any<kVec>(p.h, p.elem, row * p.cols + c, h);
      load_any<kVec>(p.weight, p.w_elem, c, w);
#pragma unroll
      for (int j = 0; j < kVec; ++j) dot += g[j] * w[j] * (h[j] * r);
    }
    // alternating buffers: the previous row's sums have been read by then
    const float mean = block_sum(dot, part[k & 1]) / static_cast<float>(p.cols);
    for (int64_t c = threadIdx.x * kVec; c < p.cols; c += step) {
      float g[kVec], h[kVec], w[kVec], d[kVec];
      load_any<kVec>(p.dy, p.elem, row * p.cols + c, g);
      load_any<kVec>(p.h, p.elem, row * p.cols + c, h);
      load_any<kVec>(p.weight, p.w_elem, c, w);
#pragma unroll
      for (int j = 0; j < kVec; ++j) d[j] = 0.0f;
      if (p.dh) load_any<kVec>(p.dh, p.elem, row * p.cols + c, d);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float xh = h[j] * r;
        acc[c + j] = (k == 0 ? 0.0f : acc[c + j]) + g[j] * xh;
        d[j] += r * (g[j] * w[j] - xh * mean);
      }
      store_any<kVec>(p.dx, p.elem, row * p.cols + c, d);
    }
  }
}

// dw = the sum of the partial rows, in their order.
__global__ void __launch_bounds__(128)
rmsnorm_dweight_kernel(const float* __restrict__ partial, int64_t parts, int64_t cols,
                       void* __restrict__ dweight, int w_elem) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
  if (c >= cols) return;
  float s = 0.0f;
  for (int64_t i = 0; i < parts; ++i) s += partial[i * cols + c];
  const float v[1] = {s};
  store_any<1>(dweight, w_elem, c, v);
}

int threads_for(int64_t cols, int vec) {
  const int64_t chunks = (cols + vec - 1) / vec;
  return static_cast<int>(std::min<int64_t>(512, (chunks + 31) / 32 * 32));
}

}  // namespace

cudaError_t launch_rmsnorm_fwd(const NormFwdCall& c) {
  const FwdArgs a = {c.x, c.residual, c.weight, c.h, c.y, c.scale, c.rstd, c.cols,
                     c.x_elem, c.h_elem, c.w_elem, c.y_elem, c.y_fp8 ? 1 : 0, c.eps};
  const unsigned grid = static_cast<unsigned>(c.rows);
  if (c.cols % 8 == 0)
    rmsnorm_fwd_long_kernel<8><<<grid, threads_for(c.cols, 8), 0, c.st>>>(a);
  else
    rmsnorm_fwd_long_kernel<1><<<grid, threads_for(c.cols, 1), 0, c.st>>>(a);
  return cudaGetLastError();
}

// Rows of the workspace: one per CTA of the backward.
int64_t rmsnorm_bwd_parts(int64_t rows, int64_t) { return std::min<int64_t>(rows, 304); }

cudaError_t launch_rmsnorm_bwd(const NormBwdCall& c) {
  const BwdArgs a = {c.dy, c.h, c.dh, c.weight, c.rstd, c.dx, c.partial, c.rows, c.cols,
                     c.elem, c.w_elem};
  const int64_t parts = rmsnorm_bwd_parts(c.rows, c.cols);
  if (c.cols % 8 == 0)
    rmsnorm_bwd_long_kernel<8><<<static_cast<unsigned>(parts), threads_for(c.cols, 8), 0, c.st>>>(a);
  else
    rmsnorm_bwd_long_kernel<1><<<static_cast<unsigned>(parts), threads_for(c.cols, 1), 0, c.st>>>(a);
  if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
  rmsnorm_dweight_kernel<<<static_cast<unsigned>((c.cols + 127) / 128), 128, 0, c.st>>>(
      c.partial, parts, c.cols, c.dweight, c.w_elem);
  return cudaGetLastError();
}

}  // namespace nf4
