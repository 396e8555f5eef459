// Uniform 4-bit weights in groups of 32, 64 or 128 along a row, each with a
// 16-bit scale and (optionally) a zero point: quantization, dequantization and
// products of few tokens. include/nf4gemm.h states the format.
#include <algorithm>

#include "gated.cuh"
#include "tc.cuh"

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

// ------------------------------------------------------------- products --
// Y[m, n] = sum over groups of s[n, j] sum_{k in j} (q[n, k] - z[n, j]) x[m, k],
// alone or (kMats = 2) for two weights whose sums meet as act(G) U.
//
// The weight's bytes bound it: half a byte a weight, read once for every 16
// tokens. The weight's rows are the 16 rows of mma.sync.m16n8k16, the tokens
// its 8 columns (one or two tiles). Nothing is rounded on the way: a code
// becomes the number 128 + q (bf16) or 1024 + q (fp16) by putting its four bits
// into the mantissa, the same number with the zero point is subtracted, and
// (q - z) x is exact in the fp32 sum; a group's sums are multiplied by its scale
// in fp32 and added to the row's.
//  * A warp has 16 rows and takes 128-wide chunks of them, kChunks neighbouring
//    ones a round: lane (g, t) loads 16 bytes (32 codes) of rows g and g + 8 a
//    chunk, straight into registers; while a chunk is multiplied, the same chunk
//    of the next round is on its way.
//  * The order of k within a chunk is free as long as both operands agree. Bits
//    of a code word are taken in pairs 16 bits apart, (e1, e5), (e0, e4),
//    (e3, e7), (e2, e6) for elements e0 to e7 of 4 bytes, and the tokens are
//    staged in shared memory in that order, 16 bytes a lane.
//  * The four lanes of a row feed one MMA, so that they have to hold codes of one
//    group. With groups of 64 and 32 they exchange words first (2 and 4 shuffles
//    for 32 codes; loads of 8 and 4 bytes instead would take 2 and 4 times the
//    load instructions).
//  * A CTA of 8 warps is kParts parts of the reduction x 8 / kParts row groups;
//    with few rows and long reductions a cluster of up to 8 CTAs splits the
//    reduction further. Every warp leaves its sums in shared memory of the CTA
//    that owns the rows, which adds them in a fixed order: repeatable, no
//    workspace.
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

struct Int4Args {
  const uint16_t* x;             // [M, K]
  const uint8_t* codes[2];
  const uint16_t* scale[2];
  const uint8_t* zero[2];        // or null
  int64_t M, N, K;
  int groups;                    // of a row
  int rounds;                    // of a row
  int window;                    // rounds whose tokens are staged at once
  int inbox;                     // bytes of shared memory for them
  int parts_log, splits, m_tiles;
  bool scale_bf16;
  Curve curve;
  void* y;
  int y_elem;
  bool accumulate;
};

// y[i] = v (+ y[i]), of type `elem`.
__device__ __forceinline__ void store_sum(void* y, int elem, int64_t i, float v, bool accumulate) {
  if (elem == kElemF32) {
    float* o = static_cast<float*>(y) + i;
    *o = accumulate ? v + *o : v;
  } else if (elem == kElemBf16) {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(y) + i;
    *o = __float2bfloat16_rn(accumulate ? v + __bfloat162float(*o) : v);
  } else {
    __half* o = static_cast<__half*>(y) + i;
    *o = __float2half_rn(accumulate ? v + __half2float(*o) : v);
  }
}

__device__ __forceinline__ uint4 load_codes(const uint8_t* p, bool in) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (in)
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
  return v;
}

template <bool kF16>
__device__ __forceinline__ void mma_16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Codes 4 bits wide in bits 0-3 and 16-19 of w as two numbers less the zero
// point's (zz: the same two numbers made of it).
template <bool kF16>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t zz) {
  constexpr uint32_t kOne = kF16 ? 0x64006400u : 0x43004300u;     // 1024, 128
  const uint32_t v = (w & 0x000f000fu) | kOne;
  if constexpr (kF16) {
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&zz));
    return *reinterpret_cast<const uint32_t*>(&d);
  } else {
    const __nv_bfloat162 d =
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&zz));
    return *reinterpret_cast<const uint32_t*>(&d);
  }
}

// The four lanes' words of a row, exchanged so that word w of every lane is of
// the chunk's group w kPer / 4 (kPer groups a chunk).
template <int kPer>
__device__ __forceinline__ void exchange(uint4& q, int t) {
  if constexpr (kPer >= 2) {
    const bool low = t < 2;
    const uint32_t a = __shfl_xor_sync(0xffffffffu, low ? q.z : q.x, 2);
    const uint32_t b = __shfl_xor_sync(0xffffffffu, low ? q.w : q.y, 2);
    if (low) {
      q.z = a;
      q.w = b;
    } else {
      q.x = a;
      q.y = b;
    }
  }
  if constexpr (kPer == 4) {
    const bool even = (t & 1) == 0;
    const uint32_t a = __shfl_xor_sync(0xffffffffu, even ? q.y : q.x, 1);
    const uint32_t b = __shfl_xor_sync(0xffffffffu, even ? q.w : q.z, 1);
    if (even) {
      q.y = a;
      q.w = b;
    } else {
      q.x = a;
      q.z = b;
    }
  }
}

// Lane and word that hold the run of 8 values kk (a multiple of 8) of a chunk:
// the inverse of exchange().
template <int kPer>
__device__ __forceinline__ int run_slot(int kk) {       // 4 word + lane
  const int run = kk >> 3;                               // 0 to 15
  if constexpr (kPer == 1) return 4 * (run & 3) + (run >> 2);
  else if constexpr (kPer == 2) return 4 * (2 * (run >> 3) + (run & 1)) + ((run >> 2) & 1) + (run & 2);
  else return 4 * (run >> 2) + (run & 3);
}

template <bool kF16, int kGroup, int kMats, int kNT>
__global__ void __launch_bounds__(kThreads, 2) int4_matmul_kernel(const __grid_constant__ Int4Args p) {
  constexpr int kPer = 128 / kGroup;           // groups of a chunk
  constexpr int kChunks = 4 / kMats;           // of a round
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int parts = 1 << p.parts_log, part = warp & (parts - 1), rgroup = warp >> p.parts_log;
  const int rows_cta = 16 * (kWarps >> p.parts_log);
  const int rank = static_cast<int>(blockIdx.x) % p.splits;
  const int tile = static_cast<int>(blockIdx.x) / p.splits;
  const int64_t m0 = static_cast<int64_t>(tile % p.m_tiles) * (8 * kNT);
  const int64_t row0 = static_cast<int64_t>(tile / p.m_tiles) * rows_cta;
  const int mt = static_cast<int>(min(static_cast<int64_t>(8 * kNT), p.M - m0));
  const int r_first = static_cast<int>(static_cast<int64_t>(p.rounds) * rank / p.splits);
  const int r_last = static_cast<int>(static_cast<int64_t>(p.rounds) * (rank + 1) / p.splits);
  let_next_start();
  if (p.splits > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  wait_for_previous();

  // rows past the end read the last one; their sums are dropped
  const int64_t ra = min(row0 + 16 * rgroup + g, p.N - 1), rb = min(row0 + 16 * rgroup + g + 8, p.N - 1);
  uint4 q[kMats][kChunks][2];
  uint32_t sz[kMats][2][kPer], next_sz[kMats][2][kPer];    // scale, zero point in bits 16 and up
  auto load_chunk = [&](int r, int i) {
    const int64_t k = (static_cast<int64_t>(r) * kChunks + i) * 128 + 32 * t;
#pragma unroll
    for (int mat = 0; mat < kMats; ++mat) {
      q[mat][i][0] = load_codes(p.codes[mat] + (ra * p.K + k) / 2, k < p.K);
      q[mat][i][1] = load_codes(p.codes[mat] + (rb * p.K + k) / 2, k < p.K);
    }
  };
  // lane t loads those of the round's chunk t, which the others take by shuffles
  auto load_scales = [&](int r, uint32_t (&to)[kMats][2][kPer]) {
#pragma unroll
    for (int mat = 0; mat < kMats; ++mat)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int at = (r * kChunks + t % kChunks) * kPer + j;
          const int64_t i = (h ? rb : ra) * p.groups + at;
          uint32_t v = 0x80000u;
          if (at < p.groups) {
            v = __ldg(p.scale[mat] + i);
            v |= p.zero[mat] ? static_cast<uint32_t>(__ldg(p.zero[mat] + i)) << 16 : 0x80000u;
          }
          to[mat][h][j] = v;
        }
  };

  float acc[kMats][kNT][4] = {};
  const uint4* xs = reinterpret_cast<const uint4*>(smem);
  for (int w0 = r_first; w0 < r_last; w0 += p.window) {
    const int w1 = min(w0 + p.window, r_last);
    int r = w0 + part;
    if (r < w1) {
#pragma unroll
      for (int i = 0; i < kChunks; ++i) load_chunk(r, i);
      load_scales(r, sz);
    }
    // the window's tokens, [chunk][word][token][lane]
    const int runs = (w1 - w0) * kChunks * 16;
    for (int i = threadIdx.x; i < runs * mt; i += kThreads) {
      const int tok = i / runs, run = i - tok * runs;
      const int64_t k = static_cast<int64_t>(w0) * kChunks * 128 + 8 * run;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (k < p.K) v = __ldg(reinterpret_cast<const uint4*>(p.x + (m0 + tok) * p.K + k));
      const int slot = run_slot<kPer>((8 * run) & 127);
      reinterpret_cast<uint4*>(smem)[(((run >> 4) * 4 + (slot >> 2)) * mt + tok) * 4 + (slot & 3)] =
          make_uint4(__byte_perm(v.x, v.z, 0x7632), __byte_perm(v.x, v.z, 0x5410),
                     __byte_perm(v.y, v.w, 0x7632), __byte_perm(v.y, v.w, 0x5410));
    }
    __syncthreads();
    for (; r < w1; r += parts) {
      const bool more = r + parts < w1;
      if (more) load_scales(r + parts, next_sz);
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const uint4* xc = xs + ((r - w0) * kChunks + i) * 16 * mt + 4 * g + t;
#pragma unroll
        for (int mat = 0; mat < kMats; ++mat) {
          exchange<kPer>(q[mat][i][0], t);
          exchange<kPer>(q[mat][i][1], t);
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          uint32_t za[kMats], zb[kMats];
          float sa[kMats], sb[kMats];
#pragma unroll
          for (int mat = 0; mat < kMats; ++mat) {
            const uint32_t va = __shfl_sync(0xffffffffu, sz[mat][0][j], (lane & 28) + i);
            const uint32_t vb = __shfl_sync(0xffffffffu, sz[mat][1][j], (lane & 28) + i);
            constexpr uint32_t kOne = kF16 ? 0x64006400u : 0x43004300u;
            za[mat] = kOne + (va >> 16) * 0x10001u;
            zb[mat] = kOne + (vb >> 16) * 0x10001u;
            sa[mat] = scale_value(va & 0xffffu, p.scale_bf16);
            sb[mat] = scale_value(vb & 0xffffu, p.scale_bf16);
          }
          float sum[kMats][kNT][4] = {};
#pragma unroll
          for (int w = j * (4 / kPer); w < (j + 1) * (4 / kPer); ++w) {
            uint4 x[kNT];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
              x[nt] = make_uint4(0u, 0u, 0u, 0u);
              if (8 * nt + g < mt) x[nt] = xc[(w * mt + 8 * nt) * 4];
            }
#pragma unroll
            for (int mat = 0; mat < kMats; ++mat) {
              const uint4 &qa = q[mat][i][0], &qb = q[mat][i][1];
              const uint32_t wa = w == 0 ? qa.x : w == 1 ? qa.y : w == 2 ? qa.z : qa.w;
              const uint32_t wb = w == 0 ? qb.x : w == 1 ? qb.y : w == 2 ? qb.z : qb.w;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t a[4] = {code_pair<kF16>(wa >> (8 * h), za[mat]), code_pair<kF16>(wb >> (8 * h), zb[mat]),
                                       code_pair<kF16>(wa >> (8 * h + 4), za[mat]),
                                       code_pair<kF16>(wb >> (8 * h + 4), zb[mat])};
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
                  mma_16<kF16>(sum[mat][nt], a, h ? x[nt].z : x[nt].x, h ? x[nt].w : x[nt].y);
              }
            }
          }
#pragma unroll
          for (int mat = 0; mat < kMats; ++mat)
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[mat][nt][e] = fmaf(e < 2 ? sa[mat] : sb[mat], sum[mat][nt][e], acc[mat][nt][e]);
        }
        if (more) load_chunk(r + parts, i);
      }
      if (more)
#pragma unroll
        for (int mat = 0; mat < kMats; ++mat)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < kPer; ++j) sz[mat][h][j] = next_sz[mat][h][j];
    }
    if (w1 < r_last) __syncthreads();        // the tokens may be overwritten
  }

  // every warp's sums to the CTA that owns the rows: [split, part][weight][token][row]
  const int own = rows_cta / p.splits, own_log = 31 - __clz(own);
  const uint32_t inbox = tc::smem_addr(smem) + p.inbox;
  if (p.splits > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // every CTA runs
#pragma unroll
  for (int mat = 0; mat < kMats; ++mat)
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tok = 8 * nt + 2 * t + (e & 1), row = 16 * rgroup + g + 8 * (e >> 1);
        if (tok >= mt) continue;
        const uint32_t at = inbox + 4u * ((((rank * parts + part) * kMats + mat) * mt + tok) * own + (row & (own - 1)));
        if (p.splits > 1)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(tc::mapa(at, row >> own_log)), "f"(acc[mat][nt][e])
                       : "memory");
        else
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(acc[mat][nt][e]) : "memory");
      }
  if (p.splits > 1) tc::cluster_sync();
  else __syncthreads();
  const float* sums = reinterpret_cast<const float*>(smem + p.inbox);
  for (int e = threadIdx.x; e < mt * own; e += kThreads) {
    const int tok = e >> own_log, row = e & (own - 1);
    const int64_t n = row0 + rank * own + row;
    if (n >= p.N) continue;
    float y[kMats] = {};
    for (int k = 0; k < p.splits * parts; ++k)
#pragma unroll
      for (int mat = 0; mat < kMats; ++mat) y[mat] += sums[((k * kMats + mat) * mt + tok) * own + row];
    const float v = kMats == 2 ? gated(y[0], y[kMats - 1], p.curve) : y[0];
    store_sum(p.y, p.y_elem, (m0 + tok) * p.N + n, v, p.accumulate);
  }
}

// Launch shape of a call. Estimated time, in ns: a round (16 rows x 512 codes of
// one weight or 256 of two, 4 KB a warp) takes 0.7 us alone and 1.43 us at HBM's
// rate on a full GPU (16 warps an SM); a CTA stages its tokens at 40 bytes a ns
// beside its neighbour; start and end take 1.5 us, a cluster 0.8 us more.
struct Int4Shape {
  int parts_log, splits, window;
};
constexpr int kMostStaged = 96 * 1024;        // two CTAs an SM, with their inboxes

Int4Shape plan_int4(int64_t N, int rounds, int tokens, int mats, int64_t m_tiles, int sms) {
  const int64_t round_bytes = static_cast<int64_t>(4 / mats) * 256 * tokens;
  Int4Shape best = {};
  int64_t best_cost = INT64_MAX;
  for (int pl = 3; pl >= 0; --pl)
    for (int s = 1; s <= 8 && s <= rounds && s <= 16 * (kWarps >> pl); s *= 2) {
      const int64_t rows = 16 * (kWarps >> pl), ctas = (N + rows - 1) / rows * s * m_tiles;
      const int64_t slice = (rounds + s - 1) / s, window = std::min<int64_t>(slice, kMostStaged / round_bytes);
      const int64_t windows = (slice + window - 1) / window;
      const int64_t each = (window + (1 << pl) - 1) >> pl;             // rounds of a warp and window
      const int64_t slots = 2 * static_cast<int64_t>(sms), waves = (ctas + slots - 1) / slots;
      const int64_t round = std::max<int64_t>(700, 1430 * std::min(ctas, slots) / slots);
      const int64_t cost = waves * (windows * each * round + slice * round_bytes / 40 + (windows - 1) * 700 + 1500) +
                           (s > 1 ? 800 : 0);
      if (cost < best_cost) {
        best_cost = cost;
        best = {pl, s, static_cast<int>(window)};
      }
    }
  return best;
}

template <bool kF16, int kGroup, int kMats, int kNT>
cudaError_t launch_int4_as(const Int4Call& c) {
  Int4Args a = {};
  a.x = static_cast<const uint16_t*>(c.x);
  for (int i = 0; i < 2; ++i) {
    a.codes[i] = c.w[i].codes;
    a.scale[i] = static_cast<const uint16_t*>(c.w[i].scale);
    a.zero[i] = c.w[i].zero;
  }
  a.M = c.M;
  a.N = c.w[0].rows;
  a.K = c.w[0].cols;
  a.groups = static_cast<int>(a.K / kGroup);
  constexpr int64_t kRound = 4 / kMats * 128;
  a.rounds = static_cast<int>((a.K + kRound - 1) / kRound);
  const int64_t m_tiles = (c.M + 8 * kNT - 1) / (8 * kNT);
  const int tokens = static_cast<int>(std::min<int64_t>(c.M, 8 * kNT));
  const Int4Shape shape = plan_int4(a.N, a.rounds, tokens, kMats, m_tiles, c.num_sms);
  const int64_t rows = 16 * (kWarps >> shape.parts_log);
  const int64_t grid = (a.N + rows - 1) / rows * m_tiles * shape.splits;
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  a.window = shape.window;
  a.inbox = shape.window * (4 / kMats) * 256 * tokens;
  a.parts_log = shape.parts_log;
  a.splits = shape.splits;
  a.m_tiles = static_cast<int>(m_tiles);
  a.scale_bf16 = c.w[0].scale_elem == kElemBf16;
  a.curve = c.curve;
  a.y = c.y;
  a.y_elem = c.y_elem;
  a.accumulate = c.accumulate;
  constexpr int kInbox = kWarps * 16 * kMats * 8 * kNT * 4;
  static std::once_flag once[kOnceDevices];
  once_per_device(once, c.device, [] {
    cudaFuncSetAttribute(int4_matmul_kernel<kF16, kGroup, kMats, kNT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         kMostStaged + kInbox);
  });
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(a.inbox) + kWarps * 16 * kMats * tokens * 4;
  cfg.stream = c.st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(shape.splits);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = shape.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, int4_matmul_kernel<kF16, kGroup, kMats, kNT>, a);
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
  return with_group(c.w[0].group, [&](auto g) {
    constexpr int kGroup = decltype(g)::value;
    auto go = [&](auto f16, auto mats) {
      constexpr bool kF16 = decltype(f16)::value;
      constexpr int kMats = decltype(mats)::value;
      return c.M <= 8 ? launch_int4_as<kF16, kGroup, kMats, 1>(c) : launch_int4_as<kF16, kGroup, kMats, 2>(c);
    };
    if (c.x_f16) {
      if (c.gated) return go(std::true_type{}, std::integral_constant<int, 2>{});
      return go(std::true_type{}, std::integral_constant<int, 1>{});
    }
    if (c.gated) return go(std::false_type{}, std::integral_constant<int, 2>{});
    return go(std::false_type{}, std::integral_constant<int, 1>{});
  });
}

}  // namespace nf4
