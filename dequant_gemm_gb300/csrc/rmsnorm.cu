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

// Runs of 8 elements. Where a row's length is a multiple of 8 its runs start at
// its first element; otherwise (kShift) rows start anywhere, and the runs are
// those of the whole tensor, on 16-byte boundaries: a row's first run starts
// up to 7 elements before it and its last may end behind it. `col` is the
// column of the run's first element, `at` its index in the tensor of `total`
// elements. What a run holds of the neighbouring rows is loaded with it and
// dropped (eight guarded loads of single elements took as many round trips
// to memory), and never written.
template <bool kShift>
__device__ __forceinline__ bool whole_run(int col, int cols) {
  return kShift ? col >= 0 && col + 8 <= cols : col < cols;
}
template <bool kShift>
__device__ __forceinline__ bool any_of_run(int col, int cols) {
  return kShift ? col + 8 > 0 && col < cols : col < cols;
}

template <bool kShift>
__device__ __forceinline__ void load_run(const void* p, int elem, int64_t at, int col, int cols,
                                         int64_t total, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  if (!any_of_run<kShift>(col, cols)) return;
  if (!kShift || at + 8 <= total) {
    load_any<8>(p, elem, at, v);
  } else {                           // the tensor's last run
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + j >= 0 && col + j < cols) {
        float u[1];
        load_any<1>(p, elem, at + j, u);
        v[j] = u[0];
      }
  }
}

// Drops what lies outside the row; after all loads have gone out, so that none
// is waited for before the next.
template <bool kShift>
__device__ __forceinline__ void trim_run(int col, int cols, float (&v)[8]) {
  if (!kShift || whole_run<kShift>(col, cols)) return;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (col + j < 0 || col + j >= cols) v[j] = 0.0f;
}

// A run as it lies in memory (16 or 32 bytes), so that a row on its way costs
// no more registers than it has bytes.
template <int kElem>
struct Raw {
  static constexpr int kWords = 2 * Elem<kElem>::kBytes;
  uint32_t w[kWords];

  template <bool kShift>
  __device__ __forceinline__ void load(const void* p, int64_t at, int col, int cols, int64_t total) {
#pragma unroll
    for (int j = 0; j < kWords; ++j) w[j] = 0u;
    if (!any_of_run<kShift>(col, cols)) return;
    if (!kShift || at + 8 <= total) {
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + at * Elem<kElem>::kBytes);
#pragma unroll
      for (int j = 0; j < kWords / 4; ++j) {
        const uint4 u = q[j];
        w[4 * j] = u.x;
        w[4 * j + 1] = u.y;
        w[4 * j + 2] = u.z;
        w[4 * j + 3] = u.w;
      }
    } else {                         // the tensor's last run
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j >= 0 && col + j < cols) {
          if constexpr (kElem == kElemF32) w[j] = static_cast<const uint32_t*>(p)[at + j];
          else w[j >> 1] |= static_cast<uint32_t>(static_cast<const uint16_t*>(p)[at + j]) << (16 * (j & 1));
        }
    }
  }
  // As trim_run.
  template <bool kShift>
  __device__ __forceinline__ void trim(int col, int cols) {
    if (!kShift || whole_run<kShift>(col, cols)) return;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + j < 0 || col + j >= cols) {
        if constexpr (kElem == kElemF32) w[j] = 0u;
        else w[j >> 1] &= (j & 1) ? 0xffffu : 0xffff0000u;
      }
  }
  __device__ __forceinline__ float at(int j) const {
    if constexpr (kElem == kElemF32) return __uint_as_float(w[j]);
    const float2 f = unpack2<kElem>(w[j >> 1]);
    return (j & 1) ? f.y : f.x;
  }
};

// Eight consecutive elements of a vector over the columns, zeros outside it.
// Unaligned with kShift: single elements at indexes held within the vector, so
// that the loads need no guards and go out together, or for fp32 the three
// aligned quadruples around them (single elements lie 32 bytes apart between
// lanes, and cost eight times the wavefronts).
template <int kElem>
__device__ __forceinline__ void load8_clamped(const void* p, int col, int cols, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = to_float<kElem>(static_cast<const typename Elem<kElem>::T*>(p)[min(max(col + j, 0), cols - 1)]);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (col + j < 0 || col + j >= cols) v[j] = 0.0f;
}

template <bool kShift>
__device__ __forceinline__ void load_weight(const void* p, int elem, int col, int cols, float (&v)[8]) {
  if constexpr (!kShift) {
    load_run<false>(p, elem, col, col, cols, cols, v);
  } else if (elem == kElemF32) {
    const int q = col & ~3, m = col & 3;           // m: the same in the whole row
    if (q >= 0 && q + 12 <= cols) {
      const float4* w = reinterpret_cast<const float4*>(static_cast<const float*>(p) + q);
      const float4 a = w[0], b = w[1], c = w[2];
      const float f[12] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = m == 0 ? f[j] : m == 1 ? f[j + 1] : m == 2 ? f[j + 2] : f[j + 3];
    } else {
      load8_clamped<kElemF32>(p, col, cols, v);
    }
  } else if (elem == kElemBf16) {
    load8_clamped<kElemBf16>(p, col, cols, v);
  } else {
    load8_clamped<kElemF16>(p, col, cols, v);
  }
}

template <bool kShift>
__device__ __forceinline__ void store_run(void* p, int elem, int64_t at, int col, int cols,
                                          const float (&v)[8]) {
  if (whole_run<kShift>(col, cols)) {
    store_any<8>(p, elem, at, v);
  } else if (kShift) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + j >= 0 && col + j < cols) {
        const float u[1] = {v[j]};
        store_any<1>(p, elem, at + j, u);
      }
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

// One CTA a row, held in registers between the sum and the output: x and the
// residual are read once, h and y written once. A thread holds kNC runs of 8
// elements, blockDim.x runs apart (so that 16 lanes hold a block of the 8-bit
// output). Bound by HBM: 8192 x 4096 bf16 with an fp32 residual to e4m3 in 60 us
// (6.1 TB/s, 0.92 of the copy bandwidth; read twice it took 90). Odd lengths
// keep the 16-byte accesses (kShift): 4096 x 5119 fp32 53 us (6.3 TB/s), bf16 34
// (4.9 TB/s, by the edges' and the unaligned weight's instructions).
template <int kX, int kRes, bool kShift, int kNC>
__global__ void __launch_bounds__(1024)
rmsnorm_fwd_kernel(const FwdArgs p) {
  __shared__ float part[32];
  constexpr int kH = kRes == 2 ? kElemF32 : kX;    // the stream's type
  const int64_t row = blockIdx.x, row0 = row * p.cols, total = gridDim.x * p.cols;
  const int cols = static_cast<int>(p.cols), step = blockDim.x * 8;
  const int c0 = static_cast<int>(threadIdx.x) * 8 - (kShift ? static_cast<int>(row0 & 7) : 0);
  let_next_start();
  wait_for_previous();
  float v[kNC][8];
  if constexpr (!kShift) {
#pragma unroll
    for (int i = 0; i < kNC; ++i)
      load_run<false>(p.x, kX, row0 + c0 + i * step, c0 + i * step, cols, total, v[i]);
    if constexpr (kRes != 0) {
      float r[kNC][8];
#pragma unroll
      for (int i = 0; i < kNC; ++i)
        load_run<false>(p.residual, kH, row0 + c0 + i * step, c0 + i * step, cols, total, r[i]);
#pragma unroll
      for (int i = 0; i < kNC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = round_to(v[i][j] + r[i][j], kH);
    }
  } else {
    // As they lie in memory first: with conversions in these loads' branches
    // each is waited for before the next.
    Raw<kX> x[kNC];
    Raw<kH> r[kNC];
#pragma unroll
    for (int i = 0; i < kNC; ++i) x[i].template load<true>(p.x, row0 + c0 + i * step, c0 + i * step, cols, total);
#pragma unroll
    for (int i = 0; i < kNC; ++i)
      if (kRes) r[i].template load<true>(p.residual, row0 + c0 + i * step, c0 + i * step, cols, total);
#pragma unroll
    for (int i = 0; i < kNC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = x[i].at(j);
        if constexpr (kRes != 0) v[i][j] = round_to(v[i][j] + r[i].at(j), kH);
      }
  }
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < kNC; ++i) {
    trim_run<kShift>(c0 + i * step, cols, v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss += v[i][j] * v[i][j];
  }
  if constexpr (kRes != 0) {
#pragma unroll
    for (int i = 0; i < kNC; ++i)
      store_run<kShift>(p.h, kH, row0 + c0 + i * step, c0 + i * step, cols, v[i]);
  }
  const float rstd = rsqrtf(block_sum(ss, part) / static_cast<float>(cols) + p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < kNC; ++i) {
    const int c = c0 + i * step;
    const bool in = any_of_run<kShift>(c, cols);
    if (in) {
      float w[8];
      load_weight<kShift>(p.weight, p.w_elem, c, cols, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * w[j];
    }
    if (p.y_fp8) write_y<8>(p, row, c, in, v[i]);
    else store_run<kShift>(p.y, p.y_elem, row0 + c, c, cols, v[i]);
  }
}

// One CTA a row of any length, read twice: the second time h comes from where
// the first pass wrote it (each thread reads back its own elements).
template <int kVec>
__global__ void __launch_bounds__(512) rmsnorm_fwd_long_kernel(const FwdArgs p) {
  __shared__ float part[32];
  let_next_start();
  wait_for_previous();
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
  void *dx, *dweight;
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
  wait_for_previous();
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

// Rows of up to kNC runs a thread, in registers: gridDim.x CTAs take the rows
// in turn, the next row's loads under way while this one is reduced (kAhead),
// each thread's share of dw in registers until the CTA is done. That wants a
// thread's columns to be the same in all rows of its CTA: with kShift the
// rows' offsets repeat every 8 rows, and gridDim.x is a multiple of 8 (or
// every CTA has one row). One CTA alone writes dw itself.
// Measured with dh and the sum of the partial rows: 4096 x 3584 bf16 24 us (21
// of it here, 5.6 TB/s; in two passes over memory 92), 8192 x 4096 48 us; 4096 x
// 5119 49 us. The rows staged in shared memory by bulk copies instead took 31 us.
template <int kElem, bool kShift, int kNC, bool kAhead, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) rmsnorm_bwd_kernel(const BwdArgs p) {
  wait_for_previous();
  using R = Raw<kElem>;
  __shared__ float part[2][32];
  const int cols = static_cast<int>(p.cols), step = blockDim.x * 8;
  const int c0 = static_cast<int>(threadIdx.x) * 8 -
                 (kShift ? static_cast<int>((blockIdx.x * p.cols) & 7) : 0);
  const int64_t total = p.rows * p.cols;
  R dy[kNC], h[kNC], dh[kNC];
  float r = 0.0f;
  auto fetch = [&](int64_t row, R (&a)[kNC], R (&b)[kNC], R (&d)[kNC], float& rs) {
    rs = p.rstd[row];
#pragma unroll
    for (int i = 0; i < kNC; ++i) {
      const int c = c0 + i * step;
      const int64_t at = row * p.cols + c;
      a[i].template load<kShift>(p.dy, at, c, cols, total);
      b[i].template load<kShift>(p.h, at, c, cols, total);
      d[i].template load<kShift>(p.dh, at, c, p.dh ? cols : -8, total);
    }
  };
  if (kAhead) fetch(blockIdx.x, dy, h, dh, r);
  float w[kNC][8], acc[kNC][8];
#pragma unroll
  for (int i = 0; i < kNC; ++i) {
    load_weight<kShift>(p.weight, p.w_elem, c0 + i * step, cols, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
  }
  int k = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, ++k) {
    R dy2[kNC], h2[kNC], dh2[kNC];
    float r2 = 0.0f;
    if (!kAhead) fetch(row, dy, h, dh, r);
    else if (row + gridDim.x < p.rows) fetch(row + gridDim.x, dy2, h2, dh2, r2);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kNC; ++i) {
      dy[i].template trim<kShift>(c0 + i * step, cols);
      h[i].template trim<kShift>(c0 + i * step, cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float gx = dy[i].at(j) * (h[i].at(j) * r);
        dot += gx * w[i][j];
        acc[i][j] += gx;
      }
    }
    // alternating buffers: the previous row's sums have been read by then
    const float mean = block_sum(dot, part[k & 1]) / static_cast<float>(cols);
#pragma unroll
    for (int i = 0; i < kNC; ++i) {
      float d[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        d[j] = dh[i].at(j) + r * (dy[i].at(j) * w[i][j] - h[i].at(j) * r * mean);
      store_run<kShift>(p.dx, kElem, row * p.cols + c0 + i * step, c0 + i * step, cols, d);
    }
    if (kAhead) {
#pragma unroll
      for (int i = 0; i < kNC; ++i) {
        dy[i] = dy2[i];
        h[i] = h2[i];
        dh[i] = dh2[i];
      }
      r = r2;
    }
  }
#pragma unroll
  for (int i = 0; i < kNC; ++i) {
    const int c = c0 + i * step;
    void* out = gridDim.x == 1 ? p.dweight : p.partial + blockIdx.x * p.cols;
    const int elem = gridDim.x == 1 ? p.w_elem : kElemF32;
    if constexpr (!kShift) {
      if (c < cols) store_any<8>(out, elem, c, acc[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j >= 0 && c + j < cols) {
          const float u[1] = {acc[i][j]};
          store_any<1>(out, elem, c + j, u);
        }
    }
  }
}

// dw = the sum of the partial rows: 8 columns (a 32-byte sector of each row) a
// CTA, 64 threads a column, so that a thread has its few loads in flight at
// once and the loads of all columns fill the GPU; their sums in a fixed order.
// (32 columns of 32 threads each: 300 x 1001 8.3 us in all against 7.2 now, 4096 x
// 3584 25.7 against 24.8.)
constexpr int kSumThreads = 512;

__global__ void __launch_bounds__(kSumThreads)
rmsnorm_dweight_kernel(const float* __restrict__ partial, int parts, int64_t cols,
                       void* __restrict__ dweight, int w_elem) {
  __shared__ float sums[kSumThreads / 32][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 8 + (lane & 7);
  wait_for_previous();                               // the partial rows are written
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 10
    for (int i = threadIdx.x >> 3; i < parts; i += kSumThreads / 8) s += partial[i * cols + c];
  }
  s += __shfl_xor_sync(0xffffffffu, s, 8);
  s += __shfl_xor_sync(0xffffffffu, s, 16);
  if (lane < 8) sums[warp][lane] = s;
  __syncthreads();
  if (threadIdx.x < 8 && c < cols) {
    float v[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < kSumThreads / 32; ++i) v[0] += sums[i][threadIdx.x];
    store_any<1>(dweight, w_elem, c, v);
  }
}

// Runs of a row (of any length: wherever it starts), and threads for n each.
int64_t runs_of(int64_t cols) { return cols % 8 == 0 ? cols / 8 : (cols + 14) / 8; }
int threads_for(int64_t runs, int n) {
  return static_cast<int>(((runs + n - 1) / n + 31) / 32 * 32);
}

// Whether rows are held in registers: up to 1024 threads of 4 runs (forward,
// 2 with odd lengths) or 1 run (gradients; 4
// in 512 threads for 16-bit types of even length).
bool fwd_in_registers(int64_t cols) { return runs_of(cols) <= (cols % 8 == 0 ? 4096 : 2048); }
bool bwd_in_registers(int64_t cols, int elem) {
  return runs_of(cols) <= (cols % 8 == 0 && elem != kElemF32 ? 2048 : 1024);
}

template <int kX, int kRes>
cudaError_t launch_fwd(const NormFwdCall& c, const FwdArgs& a) {
  // four runs a thread, whose loads are in flight together, in CTAs small
  // enough that several rows share an SM; one where odd lengths cost
  // instructions and more warps hide them (4096 x 5119 bf16 34 us, with two runs
  // 48; 4096 x 1023 8.4 and 10.4). By the row's length alone: a row's sum, and
  // with it the row's result, does not depend on how many rows the call has (at
  // odd lengths on its place modulo 8, which shifts its runs).
  const int64_t runs = runs_of(c.cols);
  if (c.cols % 8 != 0 && runs <= 1024)
    return launch_next(rmsnorm_fwd_kernel<kX, kRes, true, 1>, c.rows, threads_for(runs, 1), c.st, a);
  if (c.cols % 8 != 0)
    return launch_next(rmsnorm_fwd_kernel<kX, kRes, true, 2>, c.rows, threads_for(runs, 2), c.st, a);
  if (runs <= 256)
    return launch_next(rmsnorm_fwd_kernel<kX, kRes, false, 2>, c.rows, threads_for(runs, 2), c.st, a);
  return launch_next(rmsnorm_fwd_kernel<kX, kRes, false, 4>, c.rows, threads_for(runs, 4), c.st, a);
}

template <int kElem, bool kShift>
cudaError_t launch_bwd(const NormBwdCall& c, const BwdArgs& a, unsigned parts) {
  const int64_t runs = runs_of(c.cols);
  if (!bwd_in_registers(c.cols, kElem))
    return launch_next(rmsnorm_bwd_long_kernel<kShift ? 1 : 8>, parts, 512, c.st, a);
  if constexpr (kElem == kElemF32) {
    // the next row on its way needs 32 more registers a thread than 1024
    // threads can have (4096 x 5119: 64 us with it, 78 without)
    if (runs <= 672)
      return launch_next(rmsnorm_bwd_kernel<kElem, kShift, 1, true, 672>, parts, threads_for(runs, 1),
                         c.st, a);
    return launch_next(rmsnorm_bwd_kernel<kElem, kShift, 1, false, 1024>, parts, threads_for(runs, 1),
                       c.st, a);
  } else {
    if constexpr (!kShift)
      if (runs > 1024)
        return launch_next(rmsnorm_bwd_kernel<kElem, false, 4, false, 512>, parts, threads_for(runs, 4),
                           c.st, a);
    return launch_next(rmsnorm_bwd_kernel<kElem, kShift, 1, true, 1024>, parts, threads_for(runs, 1),
                       c.st, a);
  }
}

}  // namespace

cudaError_t launch_rmsnorm_fwd(const NormFwdCall& c) {
  const FwdArgs a = {c.x, c.residual, c.weight, c.h, c.y, c.scale, c.rstd, c.cols,
                     c.x_elem, c.h_elem, c.w_elem, c.y_elem, c.y_fp8 ? 1 : 0, c.eps};
  if (!fwd_in_registers(c.cols))
    return launch_next(c.cols % 8 == 0 ? rmsnorm_fwd_long_kernel<8> : rmsnorm_fwd_long_kernel<1>, c.rows,
                       512, c.st, a);
  const int res = !c.residual ? 0 : c.h_elem == c.x_elem ? 1 : 2;
  auto go = [&](auto x) {
    constexpr int kX = decltype(x)::value;
    if (res == 0) return launch_fwd<kX, 0>(c, a);
    if (res == 1) return launch_fwd<kX, 1>(c, a);
    return launch_fwd<kX, 2>(c, a);
  };
  if (c.x_elem == kElemF32) return go(std::integral_constant<int, kElemF32>{});
  if (c.x_elem == kElemBf16) return go(std::integral_constant<int, kElemBf16>{});
  return go(std::integral_constant<int, kElemF16>{});
}

// CTAs of the backward, and rows of its workspace: as many as run at once, so
// that none waits for another's end (a multiple of 8: rmsnorm_bwd_kernel). An
// SM's registers hold 1024 threads of 64 (16-bit types) or 800 of 80 (fp32).
int64_t rmsnorm_bwd_parts(int64_t rows, int64_t cols, int elem, int sms) {
  const int64_t per_sm = std::clamp((elem == kElemF32 ? 800 : 1024) / threads_for(runs_of(cols), 1), 1, 8);
  return std::min(rows, std::max<int64_t>(8, sms * per_sm / 8 * 8));
}

cudaError_t launch_rmsnorm_bwd(const NormBwdCall& c) {
  const BwdArgs a = {c.dy, c.h, c.dh, c.weight, c.rstd, c.dx, c.dweight, c.partial, c.rows, c.cols,
                     c.elem, c.w_elem};
  const unsigned parts =
      static_cast<unsigned>(rmsnorm_bwd_parts(c.rows, c.cols, c.elem, std::min(c.num_sms, kGb300Sms)));
  auto go = [&](auto elem) {
    constexpr int kElem = decltype(elem)::value;
    return c.cols % 8 == 0 ? launch_bwd<kElem, false>(c, a, parts) : launch_bwd<kElem, true>(c, a, parts);
  };
  const cudaError_t e = c.elem == kElemF32 ? go(std::integral_constant<int, kElemF32>{})
                        : c.elem == kElemBf16 ? go(std::integral_constant<int, kElemBf16>{})
                                              : go(std::integral_constant<int, kElemF16>{});
  if (e != cudaSuccess || (parts == 1 && bwd_in_registers(c.cols, c.elem))) return e;
  return launch_next(rmsnorm_dweight_kernel, (c.cols + 7) / 8, kSumThreads, c.st, c.partial,
                     static_cast<int>(parts), c.cols, c.dweight, c.w_elem);
}

}  // namespace nf4
