// Shared definitions of the 8-bit floating point operators: the block-scaled
// e4m3 format, its conversions, and the launchers of the quantizer, the
// products and the RMS norm that feeds them.
//
// Format: values x of a block (1 x 128 of an activation, 128 x 128 of a
// weight; the last block of a row or column may be short) are stored as e4m3
// codes q with one fp32 scale s:
//   a = max |x|,  s = fl32(a / 448),  q = e4m3(fl32(x * fl32(1 / s)))
// (448 is the largest e4m3 value; rounding to nearest even, saturating), and
// stand for q * s. A block with a < 2^-117 has s = 0 and zero codes, so that s
// and 1 / s are always normal numbers. A NaN or an infinity in a block makes
// the whole block NaN.
#pragma once

#include "common.cuh"

namespace nf4 {

// Kernel numbers of report_status (see nf4_poll_device_status_site).
constexpr uint32_t kSiteFp8Fwd = 4, kSiteFp8Dx = 5, kSiteGatedFwd = 6, kSiteGatedDx = 7;

constexpr int kFp8Block = NF4_FP8_BLOCK;      // 128
constexpr float kE4m3Max = 448.0f;
constexpr float kFp8MinAmax = 6.018531076210112e-36f;   // 2^-117

// Scale of a block from its largest magnitude, and the factor its values are
// multiplied by (a NaN or an infinity passes through). The division by 448
// is div_by_const's, checked against the exact quotient for every significand
// (results are normal, so the exponent does not matter).
__device__ __forceinline__ float fp8_scale(float amax) {
  const float s = div_by_const<448>(amax);
  return amax < kFp8MinAmax ? 0.0f : amax <= 3.402823466e38f ? s : amax;
}
__device__ __forceinline__ float fp8_inverse(float scale) {
  return scale == 0.0f ? 0.0f : __frcp_rn(scale);
}

// Programmatic dependent launch: lets the next kernel of the stream, if it was
// launched so, be set up while this one runs; and waits until the kernels
// before this one are complete. A kernel launched so reads and writes nothing
// in global memory before the wait.
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Launches a kernel so. On the host such a launch is no dearer than a plain one
// (a product's, with its cluster attribute, 3.2 us for 4.1; a quantizer's 3.0 for
// 3.1).
template <typename... Params, typename... Args>
cudaError_t launch_next(void (*kernel)(Params...), int64_t grid, int threads, cudaStream_t st,
                        Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// max that returns NaN if either operand is NaN (fmaxf drops it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two values rounded to e4m3 (to nearest even, saturating), lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

// Two e4m3 codes widened to fp32 (exact).
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Typed loads and stores of the fp32, bf16 and fp16 element types, widened to
// and rounded from fp32: kVec consecutive elements (8, 16-byte aligned; or 1).
template <int kElem>
struct Elem;
template <>
struct Elem<kElemF32> {
  using T = float;
  static constexpr int kBytes = 4;
};
template <>
struct Elem<kElemBf16> {
  using T = __nv_bfloat16;
  static constexpr int kBytes = 2;
};
template <>
struct Elem<kElemF16> {
  using T = __half;
  static constexpr int kBytes = 2;
};

template <int kElem>
__device__ __forceinline__ float to_float(typename Elem<kElem>::T v) {
  if constexpr (kElem == kElemF32) return v;
  else if constexpr (kElem == kElemBf16) return __bfloat162float(v);
  else return __half2float(v);
}

template <int kElem>
__device__ __forceinline__ typename Elem<kElem>::T from_float(float v) {
  if constexpr (kElem == kElemF32) return v;
  else if constexpr (kElem == kElemBf16) return __float2bfloat16_rn(v);
  else return __float2half_rn(v);
}

template <int kElem>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (kElem == kElemBf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

template <int kElem>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (kElem == kElemBf16)
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// 8 consecutive elements at p + i (16-byte aligned) into v.
template <int kElem>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (kElem == kElemF32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack2<kElem>(u[j]);
      v[2 * j] = f.x;
      v[2 * j + 1] = f.y;
    }
  }
}

template <int kElem>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
  if constexpr (kElem == kElemF32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(pack2<kElem>(v[0], v[1]), pack2<kElem>(v[2], v[3]), pack2<kElem>(v[4], v[5]),
                   pack2<kElem>(v[6], v[7]));
  }
}

// One product of block-scaled e4m3 operands, as the launchers take it: the
// forward Y [M, N] = dq(A) dq(W)^T with A [M, K], or the input gradient
// dX [M, K] = dq(A) dq(W) with A [M, N]; W is [N, K].
struct Fp8Call {
  bool dx;
  const uint8_t* a;        // left operand codes [M, red], red = K (forward) or N
  const float* a_scale;    // [M, ceil(red / 128)]
  const uint8_t* w;        // weight codes [N, K]
  const float* w_scale;    // [ceil(N / 128), ceil(K / 128)]
  int64_t M, N, K;
  void* out;               // [M, N] or [M, K]
  bool out_bf16;
  bool accumulate;
  int num_sms;
  int* status;
  long long wait_limit;
  int device;
  cudaStream_t st;
};
cudaError_t launch_fp8_matmul(const Fp8Call& c);

// x_elem: NF4_F32, NF4_BF16 or NF4_F16; block_rows 1 or 128.
cudaError_t launch_fp8_quantize(const void* x, int x_elem, int64_t rows, int64_t cols,
                                int block_rows, uint8_t* codes, float* scale, cudaStream_t st);
cudaError_t launch_fp8_dequantize(const uint8_t* codes, const float* scale, int64_t rows,
                                  int64_t cols, int block_rows, void* out, int out_elem,
                                  cudaStream_t st);

// One RMS norm call: h = round(x + residual) (residual null: h = x, not
// written), rstd = 1 / sqrt(mean(h^2) + eps), y = h rstd w.
struct NormFwdCall {
  const void* x;
  int x_elem;
  const void* residual;    // null, or [rows, cols] of h_elem
  const void* weight;      // [cols] of w_elem
  int w_elem;
  void* h;                 // [rows, cols] of h_elem, with a residual only
  int h_elem;              // residual's type; x's without one
  void* y;                 // codes (fp8) or [rows, cols] of y_elem
  int y_elem;
  bool y_fp8;
  float* scale;            // fp8: [rows, ceil(cols / 128)]
  float* rstd;             // null or [rows]
  int64_t rows, cols;
  float eps;
  cudaStream_t st;
};
cudaError_t launch_rmsnorm_fwd(const NormFwdCall& c);

struct NormBwdCall {
  const void* dy;          // [rows, cols] of elem
  const void* h;           // [rows, cols] of elem
  const void* dh;          // null, or [rows, cols] of elem
  int elem;
  const void* weight;      // [cols] of w_elem
  int w_elem;
  const float* rstd;       // [rows]
  void* dx;                // [rows, cols] of elem
  void* dweight;           // [cols] of w_elem
  float* partial;          // rmsnorm_bwd_parts(rows, cols, elem, kGb300Sms) x cols
  int64_t rows, cols;
  int num_sms;
  cudaStream_t st;
};
// Partial rows of the weight's gradient on a GPU (or a part of one) of `sms` SMs;
// the workspace, whose size is asked for without a device, has room for a whole
// GB300's.
constexpr int kGb300Sms = 152;
int64_t rmsnorm_bwd_parts(int64_t rows, int64_t cols, int elem, int sms);
cudaError_t launch_rmsnorm_bwd(const NormBwdCall& c);

}  // namespace nf4
