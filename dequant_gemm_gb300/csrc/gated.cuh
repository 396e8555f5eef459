// Shared definitions of the gated feed-forward block: the activations, the
// launchers of its 8-bit kernels, and the 4-bit weights in groups.
//
//   act(g) = g sigma(p(g)),  p(g) = g (c0 + c1 g^2),  sigma(p) = 1 / (1 + exp(-p))
// SiLU is c = (1, 0); GELU in its tanh form is c = 2 sqrt(2 / pi) (1, 0.044715),
// since (1 + tanh(z)) / 2 = sigma(2 z). One code path serves both, with two
// numbers for the activation.
#pragma once

#include "fp8.cuh"

namespace nf4 {

// The exponent of 2 that sigma(p) = 1 / (1 + 2^t) takes: t = g (k0 + k1 g^2),
// k = -log2(e) c; c = -k / log2(e) for the derivative.
struct Curve {
  float k0, k1;            // k1 = 0: SiLU
  float c0, c1;
};
inline Curve curve_of(int32_t activation) {
  constexpr double kLog2e = 1.4426950408889634, kGelu = 1.5957691216057308;    // 2 sqrt(2 / pi)
  const double c0 = activation == NF4_GELU_TANH ? kGelu : 1.0;
  const double c1 = activation == NF4_GELU_TANH ? kGelu * 0.044715 : 0.0;
  return {static_cast<float>(-kLog2e * c0), static_cast<float>(-kLog2e * c1), static_cast<float>(c0),
          static_cast<float>(c1)};
}

// Two fp32 operations at once, each rounded by itself.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 both(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// max(a, |b|, |c|), NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// sigma(p(g)), by the base-2 exponential and the reciprocal of PTX (2^-22 and
// 1 ulp). The exponent's rounding makes the relative error grow with |p|, by
// 2^-23 a unit, where sigma is small (p < 0). kCubic false: k1 is 0, whatever g^2.
__device__ __forceinline__ float sigma_of(float t) {
  float e, s;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
  asm("rcp.approx.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
  return s;
}
template <bool kCubic>
__device__ __forceinline__ float gate_sigma(float g, Curve c) {
  return sigma_of(g * (kCubic ? fmaf(c.k1, g * g, c.k0) : c.k0));
}

// act(g) u
template <bool kCubic>
__device__ __forceinline__ float gated(float g, float u, Curve c) { return g * gate_sigma<kCubic>(g, c) * u; }
__device__ __forceinline__ float gated(float g, float u, Curve c) {
  return c.k1 == 0.0f ? gated<false>(g, u, c) : gated<true>(g, u, c);
}

// One gated forward as the launcher takes it: y = act(A Wg^T) * (A Wu^T).
struct GatedFwdCall {
  const uint8_t* a;                  // [M, K] codes
  const float* a_scale;              // [M, ceil(K / 128)]
  const uint8_t *wg, *wu;            // [N, K] codes
  const float *wg_scale, *wu_scale;  // [ceil(N / 128), ceil(K / 128)]
  int64_t M, N, K;
  Curve curve;
  void* y;                           // codes (fp8) or [M, N], fp32 or bf16
  bool y_fp8, y_bf16;
  float* scale;                      // fp8: [M, ceil(N / 128)]
  void *g, *u;                       // null, or bf16 [M, N]
  int num_sms;
  int* status;
  long long wait_limit;
  int device;
  cudaStream_t st;
};
cudaError_t launch_gated_fwd(const GatedFwdCall& c);

// Its input gradient: dX [M, K] = dG Wg + dU Wu.
struct GatedDxCall {
  const uint8_t *dg, *du;            // [M, N] codes
  const float *dg_scale, *du_scale;  // [M, ceil(N / 128)]
  const uint8_t *wg, *wu;
  const float *wg_scale, *wu_scale;
  int64_t M, N, K;
  void* out;
  bool out_bf16;
  bool accumulate;
  int num_sms;
  int* status;
  long long wait_limit;
  int device;
  cudaStream_t st;
};
cudaError_t launch_gated_dx(const GatedDxCall& c);

// dG and dU in 8 bits from dy (of dy_elem) and the kept bf16 g and u.
cudaError_t launch_gated_bwd(const void* dy, int dy_elem, const void* g, const void* u,
                             int64_t rows, int64_t cols, Curve curve, uint8_t* dg, float* dg_scale,
                             uint8_t* du, float* du_scale, cudaStream_t st);

// 4-bit weights in groups (include/nf4gemm.h states the format): a scale's value.
__device__ __forceinline__ float scale_value(uint32_t bits, bool bf16) {
  return bf16 ? __uint_as_float(bits << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}

cudaError_t launch_int4_quantize(const void* w, int w_elem, int64_t rows, int64_t cols, int group,
                                 bool scale_bf16, uint8_t* codes, void* scale, uint8_t* zero,
                                 cudaStream_t st);
cudaError_t launch_int4_dequantize(const nf4_int4_weight& w, void* out, int out_elem, cudaStream_t st);

// Products of few tokens with one such weight, or with two as the gated block.
struct Int4Call {
  const void* x;           // [M, K], bf16 or (x_f16) fp16
  bool x_f16;
  int64_t M;
  nf4_int4_weight w[2];
  bool gated;              // both weights
  Curve curve;
  void* y;                 // [M, N] of y_elem
  int y_elem;
  bool accumulate;
  int num_sms;
  int device;
  cudaStream_t st;
};
cudaError_t launch_int4_matmul(const Int4Call& c);

}  // namespace nf4
