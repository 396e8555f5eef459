// The gradients of the gated block's product (gated.cuh), in 8 bits for the two
// products that make the input gradient of them (fp8_gemm.cu):
//   dG = dY U act'(G), dU = dY act(G),
//   act'(g) = s + g s (1 - s) p'(g), s = sigma(p(g)), p'(g) = c0 + 3 c1 g^2
#include "gated.cuh"

namespace nf4 {
namespace {

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
