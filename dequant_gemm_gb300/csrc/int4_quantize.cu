// Quantization to uniform 4-bit weights in groups of 32, 64 or 128 along a row,
// each with a 16-bit scale and (optionally) a zero point, and back.
// include/nf4gemm.h states the format and the rounding steps.
#include <type_traits>

#include "gated.cuh"

namespace nf4 {
namespace {

// A streaming pass. 8 consecutive values a thread and step, a group in kGroup / 8
// neighbouring lanes; kQuantUnroll steps keep that many loads in flight.
//
// rint(w / s) needs the quotient as IEEE division rounds it (a tie of the rounded
// quotient is a tie). q = RN(w r) with r = RN(1 / s) is within an ulp, its remainder
// w - q s is exact in one FMA, and RN(q + rem r) is the correctly rounded quotient
// (Markstein) where nothing leaves the normal range: s >= 2^-64 (smaller scales
// divide), and quotients near a half or above, which alone matter.
// Measured at 11008 x 4096, 1, 2, 3 and 4 steps: fp32 with zero points 34.2, 32.6, 33.0
// and 33.4 us (two: 6.3 TB/s), bf16 32.3, 29.9, 30.0 and 30.9 (the arithmetic), without
// zero points 27.0, 25.9, 24.9 and 26.6. Back: bf16 19.8 us, fp32 34.0 (6.0 TB/s).
constexpr int kQuantUnroll = 2;
constexpr float kSmallScale = 5.421010862427522e-20f;     // 2^-64

template <int kElem, int kGroup, bool kZero>
__global__ void __launch_bounds__(256)
int4_quantize_kernel(const void* __restrict__ w, int64_t runs, bool bf16, uint32_t* __restrict__ codes,
                     uint16_t* __restrict__ scale, uint8_t* __restrict__ zero) {
  let_next_start();
  wait_for_previous();
  constexpr int kLanes = kGroup / 8;
  constexpr float kMagic = 12582912.0f;                    // 1.5 2^23: x + kMagic holds rint(x) in its low bits
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (256 * kQuantUnroll) + threadIdx.x;
  float v[kQuantUnroll][8];
#pragma unroll
  for (int i = 0; i < kQuantUnroll; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    if (first + 256 * i < runs) load8<kElem>(w, 8 * (first + 256 * i), v[i]);
  }
#pragma unroll
  for (int i = 0; i < kQuantUnroll; ++i) {
    const int64_t run = first + 256 * i;
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      lo = fminf(lo, kZero ? v[i][j] : -fabsf(v[i][j]));
      if (kZero) hi = fmaxf(hi, v[i][j]);
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
    int z = kZero ? 0 : 8;
    if (kZero && s != 0.0f) z = static_cast<int>(fminf(rintf(__fdiv_rn(-lo, s)), 15.0f));
    uint32_t out = 0;
    // code j of the rounded quotient's bits: the even element in the high half
    auto put = [&](int j, uint32_t bits) {
      const int code = static_cast<int>(bits) + (z - __float_as_int(kMagic));
      out |= static_cast<uint32_t>(__vimin_s32_relu(code, 15)) << (4 * (j ^ 1));
    };
    if (s >= kSmallScale) {
      const float inverse = __frcp_rn(s);
      const uint64_t r = pair_of(inverse, inverse), minus_s = pair_of(-s, -s), magic = pair_of(kMagic, kMagic);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const uint64_t x = pair_of(v[i][j], v[i][j + 1]), q = mul2(x, r);
        const uint64_t m = add2(fma2(fma2(q, minus_s, x), r, q), magic);
        put(j, static_cast<uint32_t>(m));
        put(j + 1, static_cast<uint32_t>(m >> 32));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        put(j, __float_as_uint(__fadd_rn(s == 0.0f ? 0.0f : __fdiv_rn(v[i][j], s), kMagic)));
    }
    if (run >= runs) continue;
    codes[run] = out;
    if (run % kLanes == 0) {
      scale[run / kLanes] = static_cast<uint16_t>(bits);
      if (kZero) zero[run / kLanes] = static_cast<uint8_t>(z);
    }
  }
}

// 16 bytes of values a thread and step, so that a warp's stores are whole lines.
constexpr int kDequantUnroll = 4;

template <int kElem>
__global__ void __launch_bounds__(256)
int4_dequantize_kernel(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scale,
                       const uint8_t* __restrict__ zero, int64_t runs, int group_log, bool bf16,
                       void* __restrict__ out) {
  constexpr int kRun = 16 / Elem<kElem>::kBytes;           // 4 or 8 values
  constexpr int kRunLog = kRun == 4 ? 2 : 3;
  using Codes = std::conditional_t<kRun == 4, uint16_t, uint32_t>;
  let_next_start();
  wait_for_previous();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (256 * kDequantUnroll) + threadIdx.x;
  uint32_t q[kDequantUnroll], s[kDequantUnroll], z[kDequantUnroll];
#pragma unroll
  for (int i = 0; i < kDequantUnroll; ++i) {
    const int64_t run = min(first + 256 * i, runs - 1), j = run >> (group_log - kRunLog);
    q[i] = reinterpret_cast<const Codes*>(codes)[run];
    s[i] = scale[j];
    z[i] = zero ? zero[j] : 8u;
  }
#pragma unroll
  for (int i = 0; i < kDequantUnroll; ++i) {
    if (first + 256 * i >= runs) break;
    const float f = scale_value(s[i], bf16);
    float v[kRun];
#pragma unroll
    for (int j = 0; j < kRun; ++j)      // 2^23 + n has the whole number n in its low bits: n - z is exact
      v[j] = (__uint_as_float(0x4b000000u | (q[i] >> (4 * (j ^ 1)) & 15u)) - __uint_as_float(0x4b000000u | z[i])) * f;
    uint4 w;
    if constexpr (kRun == 4)
      w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    else
      w = make_uint4(pack2<kElem>(v[0], v[1]), pack2<kElem>(v[2], v[3]), pack2<kElem>(v[4], v[5]),
                     pack2<kElem>(v[6], v[7]));
    __stcs(static_cast<uint4*>(out) + first + 256 * i, w);
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
                         (runs + 256 * kQuantUnroll - 1) / (256 * kQuantUnroll), 256, st, w, runs, scale_bf16,
                         reinterpret_cast<uint32_t*>(codes), static_cast<uint16_t*>(scale), zero);
    });
  });
}

cudaError_t launch_int4_dequantize(const nf4_int4_weight& w, void* out, int out_elem, cudaStream_t st) {
  return with_elem(out_elem, [&](auto elem) {
    constexpr int kElem = decltype(elem)::value;
    const int64_t runs = w.rows * w.cols * Elem<kElem>::kBytes / 16;
    return launch_next(int4_dequantize_kernel<kElem>, (runs + 256 * kDequantUnroll - 1) / (256 * kDequantUnroll), 256,
                       st, w.codes, static_cast<const uint16_t*>(w.scale), w.zero, runs,
                       w.group == 32 ? 5 : w.group == 64 ? 6 : 7, w.scale_elem == kElemBf16, out);
  });
}

}  // namespace nf4
