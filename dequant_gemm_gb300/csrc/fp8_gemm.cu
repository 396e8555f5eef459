// Products of block-scaled e4m3 operands (fp8.cuh):
//   forward    Y[m, n]  = sum_b sx[m, b] sw[n / 128, b] sum_{k in b} qx[m, k] qw[n, k]
//   input grad dX[m, k] = sum_b sy[m, b] sw[b, k / 128] sum_{n in b} qy[m, n] qw[n, k]
// (b: the 128-wide blocks of the reduction; the weight is frozen, so there is
// no weight gradient), and of the gated block (gated.cuh), whose two weights a
// CTA takes side by side:
//   forward    Y = act(G) * U,  G = X Wg^T,  U = X Wu^T
//   input grad dX = dG Wg + dU Wu, one reduction after the other
//
// The inner sums run on the tensor cores (tcgen05, kind::f8f6f4, fp32
// accumulators in tensor memory). The scales are fp32 and differ from block
// to block along the reduction, so no accumulator can run on across blocks:
// each block's sums go to a fresh tensor-memory buffer, and warps read them
// back, multiply by the block's scales and add them into fp32 totals held in
// registers, while the tensor cores fill the next buffer.
#include <algorithm>

#include "gated.cuh"
#include "tc.cuh"

namespace nf4 {
namespace {

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 inputs, fp32 accumulate, K = 32; kCg
// as for the 16-bit products.
template <int kCg>
__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  if constexpr (kCg == 1) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

// Instruction descriptor for kind::f8f6f4 with A and B e4m3 (format 0), fp32
// D; fields as in the 16-bit kind's.
__host__ __device__ constexpr uint32_t idesc_f8_f32(uint32_t m, uint32_t n, bool a_mn_major,
                                                    bool b_mn_major) {
  return (1u << 4) | (a_mn_major ? (1u << 15) : 0u) | (b_mn_major ? (1u << 16) : 0u) |
         ((n >> 3) << 17) | ((m >> 4) << 24);
}

// 16 consecutive 32-bit columns of this warp's lane quarter (no wait).
__device__ __forceinline__ void tmem_ld16f(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  tc::tmem_ld16(taddr, r);
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
}

// Shared-memory accesses by 32-bit address (through the realigned base pointer
// the compiler would emit generic ones).
__device__ __forceinline__ float lds(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 lds128(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// Four bytes from global to shared memory, or zeros (ok false: src is not
// read), without a register or a wait; and this thread's arrival on an mbarrier
// once all its copies so far have landed.
__device__ __forceinline__ void copy4(uint32_t dst, const float* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void arrive_on_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Arrive on an mbarrier of the cluster without ordering this thread's memory
// accesses: what it hands over is tensor memory whose reads have completed
// (tcgen05.wait::ld). The releasing form cost the reading warps 350 cycles a
// block.
__device__ __forceinline__ void arrive_relaxed(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
               : "memory");
}

// The two halves of a cluster barrier that orders nothing: a CTA's shared
// memory may be written by the others once it has started.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// acc += s * v, two at a time.
__device__ __forceinline__ void scale_add(float* acc, const float (&v)[16], float s) {
#pragma unroll
  for (int j = 0; j < 16; j += 2)
    asm volatile(
        "{\n\t.reg .b64 a, b, c;\n\t"
        "mov.b64 a, {%2, %3};\n\t"
        "mov.b64 b, {%4, %4};\n\t"
        "mov.b64 c, {%0, %1};\n\t"
        "fma.rn.f32x2 c, a, b, c;\n\t"
        "mov.b64 {%0, %1}, c;\n\t}"
        : "+f"(acc[j]), "+f"(acc[j + 1])
        : "f"(v[j]), "f"(v[j + 1]), "f"(s));
}

// What a kernel computes: bit 0, the input gradient; bit 1, the gated block's.
constexpr int kForward = 0, kInputGrad = 1, kGatedForward = 2, kGatedInputGrad = 3;
constexpr uint32_t site_of(int mode) { return kSiteFp8Fwd + static_cast<uint32_t>(mode); }
static_assert(site_of(kInputGrad) == kSiteFp8Dx && site_of(kGatedForward) == kSiteGatedFwd &&
              site_of(kGatedInputGrad) == kSiteGatedDx);

struct MatmulArgs {
  const float *a_scale, *w_scale;
  void* out;
  int64_t M, cols;         // out [M, cols]
  int rb;                  // 128-blocks of the reduction
  int64_t ws_col, ws_red;  // strides of w_scale along column and reduction blocks
  int m_units, units;      // token tiles; all tiles
  int out_bf16, accumulate;
  long long mma_wait_limit;
  int* status;
  // gated block: the up projection's operands, and the blocks of one of the
  // gradient's two reductions (rb / 2)
  const float *a_scale2, *w_scale2;
  int rb1;
  // gated forward: kept projections (bf16, or null), scales of an 8-bit output
  // (or null), activation
  void *g, *u;
  float* y_scale;
  Curve curve;
};

// ------------------------------------------------------------ pair kernel --
// Large token counts. A CTA pair (cta_group::2) computes 256 tokens x 256
// columns: each CTA stages its 128 tokens and half of the weight tile (128
// columns), and receives the sums of its tokens with all 256 columns, so that
// a block's 32 KB of operands a CTA feed 512 cycles of MMA (a single CTA
// with the same tile would stage 48 KB for them, more than shared memory
// carries besides the tensor core's own reads).
//   warp 0     copies: the block's activation and weight tiles, by TMA
//   warp 1     even CTA: the four MMAs (K = 32 each) of a block into one of
//              two 256-column buffers; odd CTA: tells the even one when its
//              copies have landed
//   warps 2-3  scales: the tokens', transposed, and the weight's into shared memory
//   warps 4-11 totals: a thread holds 128 columns of one token (lane quarter
//              warp % 4, column half (warp - 4) / 4). The token's scale times
//              the column half's is one factor a thread and block.
// The 128 totals of a thread need more registers than the launch's even share
// of 168: the first four warps give theirs up.
// The gated forward takes 128 columns of both weights a tile: the even CTA
// stages the gate's, the odd one the up projection's, and a totals thread reads
// 64 columns of each (two factors a block instead of one), so that act(G) U
// needs no exchange but the largest magnitude of an 8-bit output's block, whose
// other 64 columns are in the partner warp. Its gradient runs through the two
// operand pairs' blocks one after the other. Both are bound as the plain products,
// by a block's way through tensor memory and back. Measured (CUDA graph): forward,
// 4096 tokens, two of 11008 x 4096, 8-bit output, both projections kept, 301 us, 2.45
// PFLOP/s (two plain products 284; at the power limit 316 and 293); gradient, 2048
// tokens, the same weights, 141 us, 2.61 PFLOP/s.
// Persistent: a pair takes the tiles c, c + G, ... in turn, tokens fastest,
// and the copies and MMAs of the next tile start while one is written out.
//
// Measured: 4096 x 11008 x 4096 forward 150-154 us (2.4 PFLOP/s), 2048 x 4096 x
// 11008 gradient 80 us, at the board's power limit (1376 W, 1950 MHz). A block
// takes ~850 cycles against 512 of MMA: two buffers, each of which goes
// through its MMAs, the commit, the totals warps' reads (~400 cycles) and the
// hand-back across the pair. Tensor memory has room for no third buffer, and
// narrower tiles re-read operand A from shared memory (N = 128: 168 us).
constexpr int kPairStages = 4;
constexpr int kPairBN = 256;
constexpr int kTileBytes = 128 * 128;                  // 128 rows of one block
constexpr int kPairStageBytes = 2 * kTileBytes;
constexpr int kPairTotalWarps = 8;
constexpr int kPairThreads = 32 * (4 + kPairTotalWarps);
// registers a thread after the split: 128 x 56 + 256 x 224 = 384 x 168, the launch's own
constexpr int kPairFewRegs = 56, kPairManyRegs = 224;
static_assert(128 * kPairFewRegs + 256 * kPairManyRegs <= kPairThreads * 168, "register split");
constexpr int kBoxBytes = 32 * 128;                    // a warp's 32 rows x 128 bytes of output
constexpr int kPairOffBox = kPairStages * kPairStageBytes;
// The tokens' scales, [block][token] for 16 blocks at a time, two chunks: read
// along the rows they are stored in (a thread reading its own token's scales
// touched a line a lane, and the eight warps' 256 lines a block took longer
// than half of its MMAs). The pitch of 130 keeps both the transposed stores
// (16 blocks x 2 tokens a warp) and the reads free of bank conflicts.
constexpr int kScaleChunk = 16;
constexpr int kScalePitch = 130;
constexpr int kScaleBytes = kScaleChunk * kScalePitch * 4;
constexpr int kPairOffScale = kPairOffBox + 2 * kPairTotalWarps * kBoxBytes;
// largest magnitudes, [tile parity][totals warp][lane]
constexpr int kPairOffMax = kPairOffScale + 2 * kScaleBytes;
constexpr int kMaxBytes = kPairTotalWarps * 32 * 4;
constexpr int kPairOffBars = kPairOffMax + 2 * kMaxBytes;
constexpr int kPairSmem = kPairOffBars + 256 + 1024;   // + alignment slack
static_assert(kPairSmem <= 227 * 1024, "shared memory");

// Operands as the kernels copy them: `a2` and `w2` of the up projection, `g`
// and `u` the kept projections.
template <int kMode>
struct PairMaps {
  CUtensorMap a, w, out;
};
template <>
struct PairMaps<kGatedForward> {
  CUtensorMap a, w, out, w2, g, u;
};
template <>
struct PairMaps<kGatedInputGrad> {
  CUtensorMap a, w, out, a2, w2;
};

template <int kMode>
__global__ void __launch_bounds__(kPairThreads, 1)
fp8_pair_kernel(const __grid_constant__ PairMaps<kMode> maps, const __grid_constant__ MatmulArgs p) {
  constexpr bool kDx = (kMode & 1) != 0;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t base = tc::smem_addr(smem), bars = base + kPairOffBars;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (kPairStages + s); };
  auto sum_bar = [&](int b) { return bars + 8u * (2 * kPairStages + b); };       // buffer's sums done
  auto read_bar = [&](int b) { return bars + 8u * (2 * kPairStages + 2 + b); };  // and read back
  auto sfull_bar = [&](int b) { return bars + 8u * (2 * kPairStages + 4 + b); };   // scale chunk
  auto sempty_bar = [&](int b) { return bars + 8u * (2 * kPairStages + 6 + b); };
  const uint32_t drain_bar = bars + 8u * (2 * kPairStages + 8);
  auto max_bar = [&](int q) { return bars + 8u * (2 * kPairStages + 9 + q); };   // two warps' maxima
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kPairOffBars + 8 * (2 * kPairStages + 13));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* copied = abort_flag + 1;             // stages that warp 0 has asked for

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_ctarank();
  const int cid = static_cast<int>(blockIdx.x >> 1), ncl = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      // the even CTA's stage is full once its own copies and the peer's have landed
      tc::mbar_init(full_bar(s), rank == 0 ? 2 : 1);
      tc::mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(sum_bar(b), 1);
      tc::mbar_init(read_bar(b), 2 * kPairTotalWarps);
      tc::mbar_init(sfull_bar(b), 64);   // the scale warps' lanes
      tc::mbar_init(sempty_bar(b), kPairTotalWarps);
    }
    tc::mbar_init(drain_bar, 1);
    for (int q = 0; q < 4; ++q) tc::mbar_init(max_bar(q), 2);
    *abort_flag = 0;
    tc::fence_barrier_init();
    tc::prefetch_tensormap(&maps.a);
    tc::prefetch_tensormap(&maps.w);
    tc::prefetch_tensormap(&maps.out);
  }
  if (warp == 1) tc::tmem_alloc<2>(tc::smem_addr(tmem_slot), 512);
  tc::fence_before_sync();
  tc::cluster_sync();                  // the peer's barriers exist before any arrival
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  let_next_start();
  wait_for_previous();

  auto fail = [&](uint32_t role) {
    report_status(p.status, kStatusTimeout, site_of(kMode), role);
    *abort_flag = 1;
    const uint32_t peer = tc::mapa(tc::smem_addr(const_cast<int*>(abort_flag)), rank ^ 1u);
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer), "r"(1u) : "memory");
  };
  auto tile_m = [&](int u) { return static_cast<int64_t>(u % p.m_units) * 256 + rank * 128; };
  const int64_t col_blocks = (p.cols + 127) / 128;
  auto tile_c = [&](int u) {
    return static_cast<int64_t>(u / p.m_units) * (kMode == kGatedForward ? kPairBN / 2 : kPairBN);
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPairFewRegs));
    if (warp == 0) {
      // The whole warp runs the loops of warps 0 and 1 on uniform values and one
      // elected lane issues, as in the 16-bit kernel.
      int gs = 0, slot = 0;
      uint32_t ph = 0;
      bool stop = false;
      for (int u = cid; u < p.units && !stop; u += ncl) {
        const int32_t m = static_cast<int32_t>(tile_m(u));
        const int32_t c = static_cast<int32_t>(tile_c(u)) +
                          (kMode == kGatedForward ? 0 : static_cast<int32_t>(rank) * 128);
        for (int i = 0; i < p.rb; ++i, ++gs) {
          if (__any_sync(0xffffffffu, *abort_flag != 0)) { stop = true; break; }
          int r = tc::mbar_wait_abortable(empty_bar(slot), ph ^ 1, abort_flag);
          r = __shfl_sync(0xffffffffu, r, 0);
          if (r != tc::kWaitDone) {
            if (lane == 0 && r == tc::kWaitTimeout) fail(kRoleProducer);
            stop = true;
            break;
          }
          const uint32_t dst = base + slot * kPairStageBytes;
          if (tc::elect_one()) {
            const CUtensorMap *a = &maps.a, *w = &maps.w;
            int r = i * 128;
            if constexpr (kMode == kGatedForward) {
              if (rank != 0) w = &maps.w2;
            } else if constexpr (kMode == kGatedInputGrad) {
              if (i >= p.rb1) {
                a = &maps.a2;
                w = &maps.w2;
                r = (i - p.rb1) * 128;
              }
            }
            tc::mbar_arrive_expect_tx(full_bar(slot), kPairStageBytes);
            tc::tma_load_2d(dst, a, r, m, full_bar(slot));
            if (kDx) tc::tma_load_2d(dst + kTileBytes, w, c, r, full_bar(slot));
            else tc::tma_load_2d(dst + kTileBytes, w, r, c, full_bar(slot));
          }
          __syncwarp();
          if (++slot == kPairStages) {
            slot = 0;
            ph ^= 1u;
          }
        }
      }
      if (lane == 0) *copied = gs;
    } else if (warp == 1) {
      int slot = 0;
      uint32_t ph = 0;
      bool stop = false;
      if (rank != 0) {
        for (int u = cid; u < p.units && !stop; u += ncl)
          for (int i = 0; i < p.rb; ++i) {
            int r = tc::mbar_wait_abortable(full_bar(slot), ph, abort_flag);
            r = __shfl_sync(0xffffffffu, r, 0);
            if (r != tc::kWaitDone) {
              if (lane == 0 && r == tc::kWaitTimeout) fail(kRoleMma);
              stop = true;
              break;
            }
            if (tc::elect_one()) tc::mbar_arrive_remote(tc::mapa(full_bar(slot), 0));
            __syncwarp();
            if (++slot == kPairStages) {
              slot = 0;
              ph ^= 1u;
            }
          }
      } else {
        const uint32_t idesc = idesc_f8_f32(256, kPairBN, false, kDx);
        const uint64_t adesc0 = tc::sw128_kmajor_desc(base);
        // input gradient: the weight tile's rows are the reduction, 128 columns
        // (one swizzled atom wide) each, 8-row groups 1 KB apart
        const uint64_t bdesc0 = kDx ? tc::sw128_mnmajor_desc(base + kTileBytes, 0, 1024)
                                    : tc::sw128_kmajor_desc(base + kTileBytes);
        constexpr uint32_t kBStep = kDx ? 32 * 128 / 16 : 2;   // 32 of the reduction
        int g = 0;
        for (int u = cid; u < p.units && !stop; u += ncl) {
          for (int i = 0; i < p.rb; ++i, ++g) {
            const int b = g & 1;
            // the operands first: the buffer is the one that is waited for
            int r = tc::mbar_spin_abortable<true>(full_bar(slot), ph, abort_flag, p.mma_wait_limit);
            if (r == tc::kWaitDone)
              r = tc::mbar_spin_abortable<true>(read_bar(b), ((g >> 1) & 1) ^ 1, abort_flag, 1ll << 31);
            r = __shfl_sync(0xffffffffu, r, 0);
            if (r != tc::kWaitDone) {
              if (lane == 0 && r == tc::kWaitTimeout) fail(kRoleMma);
              stop = true;
              break;
            }
            tc::fence_after_sync();
            const uint64_t off = static_cast<uint64_t>(slot * (kPairStageBytes >> 4));
            if (tc::elect_one()) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                mma_f8_ss<2>(tmem + 256u * b, adesc0 + off + 2u * j, bdesc0 + off + kBStep * j, idesc,
                             j != 0 ? 1u : 0u);
              tc::mma_commit<2>(empty_bar(slot));
              tc::mma_commit<2>(sum_bar(b));
            }
            __syncwarp();
            if (++slot == kPairStages) {
              slot = 0;
              ph ^= 1u;
            }
          }
        }
        if (tc::elect_one()) tc::mma_commit<2>(drain_bar);
        __syncwarp();
        if (lane == 0 && !tc::mbar_wait(drain_bar, 0)) fail(kRoleMma);
      }
    } else {
      // lane: block j of two tokens a step, one token a half-warp
      const int j = lane & 15, t0 = 2 * (warp - 2) + (lane >> 4);
      int ch = 0;
      bool stop = false;
      for (int u = cid; u < p.units && !stop; u += ncl) {
        const int64_t m0 = tile_m(u), cb = tile_c(u) / 128 + (kMode == kGatedForward ? 0 : lane >> 4);
        const int tokens = static_cast<int>(min(p.M - m0, static_cast<int64_t>(128)));
        const int rb1 = kMode == kGatedInputGrad ? p.rb1 : p.rb;      // blocks of a row of scales
        const float* src = p.a_scale + (m0 + t0) * rb1 + j;
        const float* wsrc = (kMode == kGatedForward && lane >= 16 ? p.w_scale2 : p.w_scale) + cb * p.ws_col +
                            j * p.ws_red;
        const bool w_in = cb < col_blocks;
        for (int i = 0; i < p.rb; i += kScaleChunk, ++ch) {
          int r = tc::mbar_wait_abortable(sempty_bar(ch & 1), ((ch >> 1) & 1) ^ 1, abort_flag);
          r = __shfl_sync(0xffffffffu, r, 0);
          if (r != tc::kWaitDone) {
            if (lane == 0 && r == tc::kWaitTimeout) fail(kRoleProducer);
            stop = true;
            break;
          }
          const uint32_t dst = base + kPairOffScale + (ch & 1) * kScaleBytes + j * kScalePitch * 4;
          const int n = i + j < p.rb ? tokens : 0;       // tokens to read in this lane's block
          const float *as = src + i, *ws = wsrc + i * p.ws_red;
          if constexpr (kMode == kGatedInputGrad)
            if (i + j >= rb1) {                          // the second reduction's
              as = p.a_scale2 + (m0 + t0) * rb1 + (i + j - rb1);
              ws = p.w_scale2 + cb * p.ws_col + (i + j - rb1) * p.ws_red;
            }
#pragma unroll 2
          for (int t = t0; t < 128; t += 4)
            copy4(dst + 4 * t, as + static_cast<int64_t>(t < n ? t - t0 : 0) * rb1, t < n);
          if (warp == 2) copy4(dst + 4 * (128 + (lane >> 4)), ws, n > 0 && w_in);
          arrive_on_copies(sfull_bar(ch & 1));
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");   // also after an abort
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPairManyRegs));
    const int q = warp & 3, half = (warp - 4) >> 2;
    // the thread's two runs of 64 columns, and its factor or (gated) two
    constexpr uint32_t kRun2 = kMode == kGatedForward ? 128 : 64;
    const uint32_t src = tmem + (static_cast<uint32_t>(32 * q) << 16) + (kMode == kGatedForward ? 64u : 128u) * half;
    const uint32_t box_addr = base + kPairOffBox + (warp - 4) * 2 * kBoxBytes;
    const int row = 32 * q + lane;       // token of this thread within the CTA's 128
    const uint32_t scales = base + kPairOffScale;

    int ch = 0, joined = 0;              // scale chunks; maxima exchanged with the partner warp
    const uint32_t read_remote = tc::mapa(read_bar(0), 0);
    uint32_t b = 0, sum_ph = 0;
    bool stop = false;
    for (int u = cid; u < p.units && !stop; u += ncl) {
      float acc[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) acc[j] = 0.0f;
      for (int i = 0; i < p.rb; ++i) {
        const int in = i % kScaleChunk;
        if (in == 0 && !__all_sync(0xffffffffu, tc::mbar_try_wait(sfull_bar(ch & 1), (ch >> 1) & 1))) {
          const int r = __shfl_sync(
              0xffffffffu, tc::mbar_wait_abortable(sfull_bar(ch & 1), (ch >> 1) & 1, abort_flag), 0);
          if (r != tc::kWaitDone) {
            if (lane == 0 && r == tc::kWaitTimeout) fail(kRoleCompute);
            stop = true;
            break;
          }
        }
        // the scales arrive while the block's sums are waited for
        const uint32_t sp = scales + (ch & 1) * kScaleBytes + in * (kScalePitch * 4);
        const float sa = lds(sp + 4 * row), sw = lds(sp + 4 * (128 + (kMode == kGatedForward ? 0 : half)));
        const float sw2 = kMode == kGatedForward ? lds(sp + 4 * 129) : sw;
        if (!__all_sync(0xffffffffu, tc::mbar_try_wait(sum_bar(b), sum_ph))) {
          const int r = __shfl_sync(0xffffffffu, tc::mbar_wait_abortable(sum_bar(b), sum_ph, abort_flag), 0);
          if (r != tc::kWaitDone) {
            if (lane == 0 && r == tc::kWaitTimeout) fail(kRoleCompute);
            stop = true;
            break;
          }
        }
        tc::fence_after_sync();
        // 64 columns at a time (16 at a time, the next on their way while the last
        // are added, ran 2% slower; loads of 32 columns spilled)
        float v[4][16];
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld16f(src + 256u * b + 16u * k, v[k]);
        const float s = sa * sw, s2 = sa * sw2;
        if (in == kScaleChunk - 1 || i + 1 == p.rb) {
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(sempty_bar(ch & 1));
          ++ch;
        }
        tc::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 4; ++k) scale_add(acc + 16 * k, v[k], s);
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld16f(src + 256u * b + kRun2 + 16u * k, v[k]);
        tc::tmem_wait_ld();
        tc::fence_before_sync();         // all read: the buffer is free
        if (lane == 0) arrive_relaxed(read_remote + 8u * b);
#pragma unroll
        for (int k = 0; k < 4; ++k) scale_add(acc + 64 + 16 * k, v[k], s2);
        b ^= 1u;
        sum_ph ^= b ^ 1u;
      }
      if (stop) break;
      // out: 128 columns of 32 tokens a warp, in boxes of 128 bytes a row whose
      // 16-byte chunks are swizzled by the row (no bank conflicts); rows and
      // columns past the end are dropped by the copy
      const int64_t m0 = tile_m(u) + 32 * q, m = m0 + lane;
      const int64_t c0 = tile_c(u) + (kMode == kGatedForward ? 64 : 128) * half;
      if (m0 >= p.M || (kMode != kGatedForward && c0 >= p.cols)) continue;
      if (kMode != kGatedForward && p.accumulate && m < p.M) {
#pragma unroll
        for (int j = 0; j < 128; j += 8) {
          if (c0 + j >= p.cols) break;
          float o[8];
          if (p.out_bf16) load8<kElemBf16>(p.out, m * p.cols + c0 + j, o);
          else load8<kElemF32>(p.out, m * p.cols + c0 + j, o);
#pragma unroll
          for (int t = 0; t < 8; ++t) acc[j + t] += o[t];
        }
      }
      auto send = [&](const CUtensorMap& map, int64_t c, int k) {
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0 && c < p.cols) {
          tc::tma_store_2d(&map, box_addr + (k & 1) * kBoxBytes, static_cast<int32_t>(c), static_cast<int32_t>(m0));
          tc::bulk_commit();
        }
      };
      auto reuse = [&] {                 // the box's previous contents have been read
        if (lane == 0) tc::bulk_wait_read_all();
        __syncwarp();
      };
      const uint32_t rowp = box_addr + 128 * lane;
      auto box16 = [&](const float* run, int k) {       // 64 columns in bf16
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float* a = run + 8 * j;
          sts128(rowp + k * kBoxBytes + 16 * (j ^ (lane & 7)), pack2<kElemBf16>(a[0], a[1]), pack2<kElemBf16>(a[2], a[3]),
                 pack2<kElemBf16>(a[4], a[5]), pack2<kElemBf16>(a[6], a[7]));
        }
      };
      auto box32 = [&](const float* run, int k) {       // 32 columns in fp32
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float* a = run + 4 * j;
          sts128(rowp + k * kBoxBytes + 16 * (j ^ (lane & 7)), __float_as_uint(a[0]), __float_as_uint(a[1]),
                 __float_as_uint(a[2]), __float_as_uint(a[3]));
        }
      };
      if constexpr (kMode == kGatedForward) {
        reuse();
        if (p.g) {
          box16(acc, 0);
          send(maps.g, c0, 0);
          box16(acc + 64, 1);
          send(maps.u, c0, 1);
        }
        if (p.curve.k1 == 0.0f) {
#pragma unroll
          for (int j = 0; j < 64; ++j) acc[j] = gated<false>(acc[j], acc[64 + j], p.curve);
        } else {
#pragma unroll
          for (int j = 0; j < 64; ++j) acc[j] = gated<true>(acc[j], acc[64 + j], p.curve);
        }
        if (p.y_scale) {
          float a = 0.0f;
#pragma unroll
          for (int j = 0; j < 64; j += 2) a = max_abs(a, acc[j], acc[j + 1]);   // columns past the end are 0
          // the other half of the block; slots by parity, since this warp may be a
          // tile ahead of the partner's read
          const uint32_t slot = base + kPairOffMax + (joined & 1) * kMaxBytes + 4 * lane;
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(slot + 128 * (warp - 4)), "f"(a) : "memory");
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(max_bar(q));
          const int r = __shfl_sync(0xffffffffu, tc::mbar_wait_abortable(max_bar(q), joined & 1, abort_flag), 0);
          if (r != tc::kWaitDone) {
            if (lane == 0 && r == tc::kWaitTimeout) fail(kRoleEpilogue);
            break;
          }
          ++joined;
          const float s = fp8_scale(max_nan(a, lds(slot + 128 * ((warp - 4) ^ 4)))), inv = fp8_inverse(s);
          if (half == 0 && m < p.M) p.y_scale[m * col_blocks + c0 / 128] = s;
          if (p.g) reuse();
          // rows of 64 bytes, their 16-byte chunks swizzled by the row's pair
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float* a8 = acc + 16 * j;
            uint32_t w[4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
              w[t] = e4m3x4(a8[4 * t] * inv, a8[4 * t + 1] * inv, a8[4 * t + 2] * inv, a8[4 * t + 3] * inv);
            sts128(box_addr + 64 * lane + 16 * (j ^ ((lane >> 1) & 3)), w[0], w[1], w[2], w[3]);
          }
          send(maps.out, c0, 0);
        } else if (p.out_bf16) {
          if (p.g) reuse();
          box16(acc, 0);
          send(maps.out, c0, 0);
        } else {
          if (p.g) reuse();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            box32(acc + 32 * h, h);
            send(maps.out, c0 + 32 * h, h);
          }
        }
      } else if (p.out_bf16) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 0) reuse();
          box16(acc + 64 * h, h);
          send(maps.out, c0 + 64 * h, h);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          if (h % 2 == 0) reuse();
          box32(acc + 32 * h, h & 1);
          send(maps.out, c0 + 32 * h, h);
        }
      }
    }
    if (lane == 0) tc::bulk_wait_all();
  }

  // neither CTA frees its tensor memory or leaves before both are done
  tc::fence_before_sync();
  tc::cluster_sync();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc<2>(tmem, 512);
    // the last commit arrives in both CTAs: the odd one stays until it has
    if (rank != 0) tc::mbar_wait(drain_bar, 0);
    // After an abort, copies in flight land before the CTA exits. The flag is
    // looked at here, where no role can set it any more: the copying warp may
    // be done before another aborts. The peer's arrival, which the even CTA's
    // barrier also counts, may not have come (the wait then runs to its limit).
    if (*abort_flag)
#pragma unroll 1
      for (int n = *copied, g = max(0, n - kPairStages); g < n; ++g)
        tc::mbar_wait(full_bar(g % kPairStages), (g / kPairStages) & 1, 1ll << 24);
  }
}

// ------------------------------------------------------------ rows kernel --
// Few tokens: the weight is what has to be read. Its 128 output columns are
// the MMA's 128 rows (A), the tokens its kBT columns (B, 16 to 128), so that
// the tensor core's and the reading warps' work shrinks with the tokens and a
// stage is a 16 KB weight tile plus kBT x 128 bytes. Tiles that do not fill
// the GPU are split along the reduction over a cluster of up to 8 CTAs, whose
// totals meet in distributed shared memory: each CTA owns kBT / S tokens,
// receives the others' totals of them and adds the S contributions in rank
// order (repeatable, no workspace, no zeroing pass).
//   warp 0 copies, warp 1 MMAs into kBufs buffers of kBT columns, warps 2-3
//   scales (the tokens', [block][token], and the tile's weight scale),
//   warps 4.. totals: a thread holds one output column for kBT / kGroups
//   tokens, whose factors it reads as broadcasts.
//
// Measured (CUDA graph): 64 tokens, 18944 x 3584, 15.6 us (4.5 TB/s; a block
// takes 0.37 us on 148 SMs, 6 TB/s of weight, and launch, first loads and the
// exchange of totals 4 us); 1 token, 4096 x 4096, 4.9 us in splits of 4.
//
// The gated forward (kMats = 2) has a tile of each weight in a stage and two
// MMAs a block, into neighbouring columns; each has its own totals warps, and
// the totals of both meet in the inbox, where act(G) U is taken. A warp then
// holds a token's 128 columns: the block of an 8-bit output. Bound by HBM: two of
// 18944 x 3584, 8-bit output, 24.0 us at one token (5.7 TB/s), 28.8 at 64; two of
// 11008 x 4096 19.1 and 24.9 (4.7 and 3.7 TB/s: 86 of 152 SMs).
template <int kBT, int kMats>
struct RowsCfg {
  static constexpr int kGroups = kBT >= 64 ? 2 : 1;      // token groups, four warps each and weight
  static constexpr int kCols = kBT / kGroups;            // tokens a thread
  static constexpr int kTotalWarps = 4 * kGroups * kMats;
  static constexpr int kThreads = 32 * (4 + kTotalWarps);
  static constexpr int kStageBytes = kMats * kTileBytes + kBT * 128;
  // what fits beside the inbox: 7 to 10 weight tiles of 16 KB in flight up to 64
  // tokens, 4 at 128, above the 35 KB an SM needs to keep HBM busy; gated 10, 6
  // at 64 tokens
  static constexpr int kStages = kMats == 2 ? (kBT == 64 ? 3 : 5)
                                            : kBT == 128 ? 4 : kBT == 64 ? 7 : kBT == 32 ? 8 : 10;
  static constexpr int kBufs = kMats * kBT == 128 ? 4 : 8;
  static constexpr int kBufCols = kMats * kBT;
  static constexpr int kTmemCols = kBufs * kBufCols;     // 128, 256, 512, 512
  static constexpr int kInboxRow = kMats * 128;          // floats of a token
  static constexpr int kPitch = kBT + 4;                 // scale row: 16-byte aligned
  static constexpr int kChunkBytes = kScaleChunk * kPitch * 4;
  static constexpr int kOffInbox = kStages * kStageBytes;
  static constexpr int kOffScale = kOffInbox + kBT * kInboxRow * 4;
  static constexpr int kOffBars = kOffScale + 2 * kChunkBytes;
  static constexpr int kNumBars = 2 * kStages + 2 * kBufs + 4 + 1;
  static constexpr int kSmem = kOffBars + 8 * kNumBars + 16 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kTmemCols <= 512, "tensor memory");
};

template <int kMode>
struct RowsMaps {
  CUtensorMap a, w;
};
template <>
struct RowsMaps<kGatedForward> {
  CUtensorMap a, w, w2;
};
template <>
struct RowsMaps<kGatedInputGrad> {
  CUtensorMap a, w, a2, w2;
};
template <int kMode, int kBT>
using RowsOf = RowsCfg<kBT, kMode == kGatedForward ? 2 : 1>;

template <int kMode, int kBT>
__global__ void __launch_bounds__((RowsOf<kMode, kBT>::kThreads), 1)
fp8_rows_kernel(const __grid_constant__ RowsMaps<kMode> maps, const __grid_constant__ MatmulArgs p) {
  constexpr bool kDx = (kMode & 1) != 0;
  constexpr int kMats = kMode == kGatedForward ? 2 : 1;
  using C = RowsOf<kMode, kBT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t base = tc::smem_addr(smem), bars = base + C::kOffBars;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (C::kStages + s); };
  auto sum_bar = [&](int b) { return bars + 8u * (2 * C::kStages + b); };
  auto read_bar = [&](int b) { return bars + 8u * (2 * C::kStages + C::kBufs + b); };
  auto sfull_bar = [&](int b) { return bars + 8u * (2 * C::kStages + 2 * C::kBufs + b); };
  auto sempty_bar = [&](int b) { return bars + 8u * (2 * C::kStages + 2 * C::kBufs + 2 + b); };
  const uint32_t drain_bar = bars + 8u * (2 * C::kStages + 2 * C::kBufs + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBars + 8 * C::kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* copied = abort_flag + 1;             // stages that warp 0 has asked for

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = static_cast<int>(gridDim.x);        // the cluster
  const int rank = static_cast<int>(blockIdx.x);
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 128, m0 = static_cast<int64_t>(blockIdx.z) * kBT;
  const int b0 = static_cast<int>(static_cast<int64_t>(p.rb) * rank / splits);
  const int nb = static_cast<int>(static_cast<int64_t>(p.rb) * (rank + 1) / splits) - b0;   // blocks here

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      tc::mbar_init(full_bar(i), 1);
      tc::mbar_init(empty_bar(i), 1);
    }
    for (int i = 0; i < C::kBufs; ++i) {
      tc::mbar_init(sum_bar(i), 1);
      tc::mbar_init(read_bar(i), C::kTotalWarps);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(sfull_bar(i), 64);
      tc::mbar_init(sempty_bar(i), C::kTotalWarps);
    }
    tc::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
    tc::prefetch_tensormap(&maps.a);
    tc::prefetch_tensormap(&maps.w);
  }
  if (warp == 1) tc::tmem_alloc<1>(tc::smem_addr(tmem_slot), C::kTmemCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  cluster_arrive();
  const uint32_t tmem = *tmem_slot;
  let_next_start();
  wait_for_previous();

  auto fail = [&](uint32_t role) {
    report_status(p.status, kStatusTimeout, site_of(kMode), role);
    *abort_flag = 1;
  };
  auto waited = [&](uint32_t bar, uint32_t parity, uint32_t role) {   // warp-uniform
    const int r = __shfl_sync(0xffffffffu, tc::mbar_wait_abortable(bar, parity, abort_flag), 0);
    if (r == tc::kWaitTimeout && lane == 0) fail(role);
    return r == tc::kWaitDone;
  };

  float acc[C::kCols];
  if (warp == 0) {
    int slot = 0;
    uint32_t ph = 0;
    int i = 0;
    for (; i < nb; ++i) {
      if (!waited(empty_bar(slot), ph ^ 1, kRoleProducer)) break;
      const uint32_t dst = base + slot * C::kStageBytes;
      int32_t k = (b0 + i) * 128;
      if (tc::elect_one()) {
        const CUtensorMap *a = &maps.a, *w = &maps.w;
        if constexpr (kMode == kGatedInputGrad) {
          if (b0 + i >= p.rb1) {
            a = &maps.a2;
            w = &maps.w2;
            k -= p.rb1 * 128;
          }
        }
        tc::mbar_arrive_expect_tx(full_bar(slot), C::kStageBytes);
        if (kDx) tc::tma_load_2d(dst, w, static_cast<int32_t>(r0), k, full_bar(slot));
        else tc::tma_load_2d(dst, w, k, static_cast<int32_t>(r0), full_bar(slot));
        if constexpr (kMats == 2)
          tc::tma_load_2d(dst + kTileBytes, &maps.w2, k, static_cast<int32_t>(r0), full_bar(slot));
        tc::tma_load_2d(dst + kMats * kTileBytes, a, k, static_cast<int32_t>(m0), full_bar(slot));
      }
      __syncwarp();
      if (++slot == C::kStages) {
        slot = 0;
        ph ^= 1u;
      }
    }
    if (lane == 0) *copied = i;
  } else if (warp == 1) {
    const uint32_t idesc = idesc_f8_f32(128, kBT, kDx, false);
    const uint64_t adesc0 = kDx ? tc::sw128_mnmajor_desc(base, 0, 1024) : tc::sw128_kmajor_desc(base);
    const uint64_t bdesc0 = tc::sw128_kmajor_desc(base + kMats * kTileBytes);
    constexpr uint32_t kAStep = kDx ? 32 * 128 / 16 : 2;   // 32 of the reduction
    int slot = 0;
    uint32_t ph = 0, buf = 0, bph = 1;
    for (int i = 0; i < nb; ++i) {
      int r = tc::mbar_spin_abortable<false>(full_bar(slot), ph, abort_flag, p.mma_wait_limit);
      if (r == tc::kWaitDone) r = tc::mbar_spin_abortable<false>(read_bar(buf), bph, abort_flag, 1ll << 31);
      r = __shfl_sync(0xffffffffu, r, 0);
      if (r != tc::kWaitDone) {
        if (lane == 0 && r == tc::kWaitTimeout) fail(kRoleMma);
        break;
      }
      tc::fence_after_sync();
      const uint64_t off = static_cast<uint64_t>(slot * (C::kStageBytes >> 4));
      if (tc::elect_one()) {
#pragma unroll
        for (int mat = 0; mat < kMats; ++mat)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_f8_ss<1>(tmem + buf * C::kBufCols + mat * kBT, adesc0 + off + mat * (kTileBytes >> 4) + kAStep * j,
                         bdesc0 + off + 2u * j, idesc, j != 0 ? 1u : 0u);
        tc::mma_commit<1>(sum_bar(buf));
        tc::mma_commit<1>(empty_bar(slot));
      }
      __syncwarp();
      if (++slot == C::kStages) {
        slot = 0;
        ph ^= 1u;
      }
      if (++buf == C::kBufs) {
        buf = 0;
        bph ^= 1u;
      }
    }
    if (tc::elect_one()) tc::mma_commit<1>(drain_bar);
    __syncwarp();
    if (lane == 0 && !tc::mbar_wait(drain_bar, 0)) fail(kRoleMma);
  } else if (warp < 4) {
    // lane: block j of two tokens a step, one token a half-warp
    const int j = lane & 15, t0 = 2 * (warp - 2) + (lane >> 4);
    const int tokens = static_cast<int>(min(p.M - m0, static_cast<int64_t>(kBT)));
    const int rb1 = kMode == kGatedInputGrad ? p.rb1 : p.rb;          // blocks of a row of scales
    const float* as0 = p.a_scale + (m0 + t0) * rb1 + b0 + j;
    const float* ws0 = (kMats == 2 && lane >= 16 ? p.w_scale2 : p.w_scale) + (r0 / 128) * p.ws_col +
                       (b0 + j) * p.ws_red;
    for (int i = 0, ch = 0; i < nb; i += kScaleChunk, ++ch) {
      if (!waited(sempty_bar(ch & 1), ((ch >> 1) & 1) ^ 1, kRoleProducer)) break;
      const uint32_t dst = base + C::kOffScale + (ch & 1) * C::kChunkBytes + j * (C::kPitch * 4);
      const int n = i + j < nb ? tokens : 0;
      const float *as = as0 + i, *ws = ws0 + i * p.ws_red;
      if constexpr (kMode == kGatedInputGrad) {
        const int b = b0 + i + j - rb1;
        if (b >= 0) {                                    // the second reduction's
          as = p.a_scale2 + (m0 + t0) * rb1 + b;
          ws = p.w_scale2 + (r0 / 128) * p.ws_col + b * p.ws_red;
        }
      }
#pragma unroll 8
      for (int t = t0; t < kBT; t += 4)
        copy4(dst + 4 * t, as + static_cast<int64_t>(t < n ? t - t0 : 0) * rb1, t < n);
      if (warp == 2 && lane < 16 * kMats) copy4(dst + 4 * (kBT + (lane >> 4)), ws, n > 0);
      arrive_on_copies(sfull_bar(ch & 1));
    }
    asm volatile("cp.async.wait_all;" ::: "memory");   // also after an abort
  } else {
    const int q = warp & 3, part = (warp - 4) / 4 % C::kGroups, mat = (warp - 4) / (4 * C::kGroups);
    const uint32_t src = tmem + (static_cast<uint32_t>(32 * q) << 16) + kBT * mat + C::kCols * part;
    const uint32_t scales = base + C::kOffScale;
    // read back into this CTA's own barrier, by its cluster address (the
    // relaxed arrival costs half of the local releasing one)
    const uint32_t read_remote = tc::mapa(read_bar(0), tc::cluster_ctarank());
#pragma unroll
    for (int j = 0; j < C::kCols; ++j) acc[j] = 0.0f;
    uint32_t buf = 0, ph = 0;
    for (int i = 0; i < nb; ++i) {
      const int in = i % kScaleChunk, ch = i / kScaleChunk;
      if (in == 0 && !waited(sfull_bar(ch & 1), (ch >> 1) & 1, kRoleCompute)) break;
      if (!waited(sum_bar(buf), ph, kRoleCompute)) break;
      tc::fence_after_sync();
      const uint32_t sp = scales + (ch & 1) * C::kChunkBytes + in * (C::kPitch * 4);
      const float w = lds(sp + 4 * (kBT + mat));
#pragma unroll
      for (int c = 0; c < C::kCols; c += 16) {
        float v[16];
        tmem_ld16f(src + C::kBufCols * buf + c, v);
        float4 f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = lds128(sp + 4 * (C::kCols * part + c) + 16 * k);
        tc::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 4; ++k) {   // the two scales first: their product may be all that is in range
          acc[c + 4 * k] = fmaf(v[4 * k], f[k].x * w, acc[c + 4 * k]);
          acc[c + 4 * k + 1] = fmaf(v[4 * k + 1], f[k].y * w, acc[c + 4 * k + 1]);
          acc[c + 4 * k + 2] = fmaf(v[4 * k + 2], f[k].z * w, acc[c + 4 * k + 2]);
          acc[c + 4 * k + 3] = fmaf(v[4 * k + 3], f[k].w * w, acc[c + 4 * k + 3]);
        }
      }
      tc::fence_before_sync();
      if (lane == 0) arrive_relaxed(read_remote + 8u * buf);
      if (in == kScaleChunk - 1 || i + 1 == nb) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(sempty_bar(ch & 1));
      }
      if (++buf == C::kBufs) {
        buf = 0;
        ph ^= 1u;
      }
    }
  }

  // totals to the CTAs that own the tokens: inbox[source][token][column]
  cluster_wait();                                  // every CTA of the cluster runs
  const int own_log = 31 - __clz(kBT / splits), own = 1 << own_log;   // tokens a CTA owns
  if (warp >= 4) {
    const int part = (warp - 4) / 4 % C::kGroups, mat = (warp - 4) / (4 * C::kGroups);
    const int col = 128 * mat + 32 * (warp & 3) + lane;
#pragma unroll
    for (int j = 0; j < C::kCols; ++j) {
      const int t = C::kCols * part + j;
      const uint32_t at = base + C::kOffInbox + 4u * ((rank * own + (t & (own - 1))) * C::kInboxRow + col);
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(tc::mapa(at, t >> own_log)), "f"(acc[j])
                   : "memory");
    }
  }
  tc::fence_before_sync();
  tc::cluster_sync();                              // every total has arrived
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc<1>(tmem, C::kTmemCols);
    if (*abort_flag)   // copies in flight land before the CTA exits, as in the pair kernel
#pragma unroll 1
      for (int n = *copied, g = max(0, n - C::kStages); g < n; ++g)
        tc::mbar_wait(full_bar(g % C::kStages), (g / C::kStages) & 1, 1ll << 24);
  }
  // own tokens x 128 columns, four columns a thread
  for (int e = threadIdx.x; e < own * 32; e += C::kThreads) {
    const int t = e >> 5, c = (e & 31) * 4;
    const int64_t m = m0 + static_cast<int64_t>(rank) * own + t;
    const int64_t o = m * p.cols + r0 + c;
    const uint32_t at = base + C::kOffInbox + 4u * (t * C::kInboxRow + c);
    auto total = [&](uint32_t first) {
      float4 y = lds128(first);
      for (int k = 1; k < splits; ++k) {
        const float4 z = lds128(first + 4u * C::kInboxRow * own * k);
        y.x += z.x;
        y.y += z.y;
        y.z += z.z;
        y.w += z.w;
      }
      return y;
    };
    if constexpr (kMats == 2) {
      if (m >= p.M) continue;                      // a whole warp's token
      const bool in = r0 + c < p.cols;
      const float4 g = total(at), u = total(at + 512);
      float4 y = make_float4(gated(g.x, u.x, p.curve), gated(g.y, u.y, p.curve), gated(g.z, u.z, p.curve),
                             gated(g.w, u.w, p.curve));
      if (in && p.g) {
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.g) + o) =
            make_uint2(pack2<kElemBf16>(g.x, g.y), pack2<kElemBf16>(g.z, g.w));
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.u) + o) =
            make_uint2(pack2<kElemBf16>(u.x, u.y), pack2<kElemBf16>(u.z, u.w));
      }
      if (p.y_scale) {
        float a = max_abs(max_abs(0.0f, y.x, y.y), y.z, y.w);   // 0 past the end
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, k));
        const float s = fp8_scale(a), inv = fp8_inverse(s);
        if (in)
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + o) =
              e4m3x4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
        if (lane == 0) p.y_scale[m * ((p.cols + 127) / 128) + r0 / 128] = s;
      } else if (in && p.out_bf16) {
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + o) =
            make_uint2(pack2<kElemBf16>(y.x, y.y), pack2<kElemBf16>(y.z, y.w));
      } else if (in) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = y;
      }
      continue;
    }
    if (m >= p.M || r0 + c >= p.cols) continue;
    float4 y = total(at);
    if (p.out_bf16) {
      uint2* out = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + o);
      if (p.accumulate) {
        const uint2 u = *out;
        const float2 a = unpack2<kElemBf16>(u.x), b = unpack2<kElemBf16>(u.y);
        y.x += a.x;
        y.y += a.y;
        y.z += b.x;
        y.w += b.y;
      }
      *out = make_uint2(pack2<kElemBf16>(y.x, y.y), pack2<kElemBf16>(y.z, y.w));
    } else {
      float4* out = reinterpret_cast<float4*>(static_cast<float*>(p.out) + o);
      if (p.accumulate) {
        const float4 a = *out;
        y.x += a.x;
        y.y += a.y;
        y.z += a.z;
        y.w += a.w;
      }
      *out = y;
    }
  }
}

// Launch attributes of both kernels: a cluster along x, and programmatic launch
// (the set-up, and the waiting for the last tiles of the kernel before, overlap).
struct LaunchAttrs {
  cudaLaunchAttribute a[2];

  void set(cudaLaunchConfig_t* cfg, int cluster) {
    a[0].id = cudaLaunchAttributeClusterDimension;
    a[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    a[0].val.clusterDim.y = 1;
    a[0].val.clusterDim.z = 1;
    a[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[1].val.programmaticStreamSerializationAllowed = 1;
    cfg->attrs = a;
    cfg->numAttrs = 2;
  }
};

// Launch shape of a rows call: splits of the reduction, and its time in 0.01
// us, start-up left out. Measured at 128 tokens a tile on the decoder shapes:
// 0.46 us a block, 1.5 us a round for the last block and the reduction (up to 64
// tokens a block takes 0.37 us, which the estimate does not tell apart).
// The gated block's kernels: a block takes the longer of its own latency and its
// share of HBM among the CTAs that run, and joining costs more the more CTAs share
// a tile. Two weights of 11008 x 4096 at 64 tokens: 25.8, 31.7, 34.1, 54.9 us in 1,
// 2, 4, 8 splits (estimated 22.6, 30.0, 29.5, 43.6 with 3 us to start); 4112 x 3600
// at one token 15.8, 11.0, 9.8, 18.2 (15.9, 10.3, 10.0, 13.5).
struct RowsPlan {
  int splits;
  int64_t cost;
};

// The operands of a call, as the launchers make tensor maps of them; a2 and w2
// the up projection's.
struct Operands {
  const uint8_t *a, *a2, *w, *w2;
  int64_t red;             // columns of a (of one reduction)
  int64_t M, N, K;         // a has M rows, the weight is [N, K]
  int num_sms, device;
  cudaStream_t st;
};

template <int kMode, int kBT>
cudaLaunchConfig_t rows_config(int splits, int64_t row_tiles, int64_t m_tiles, cudaStream_t st,
                               LaunchAttrs* attrs) {
  using C = RowsOf<kMode, kBT>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(splits), static_cast<unsigned>(row_tiles),
                     static_cast<unsigned>(m_tiles));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  attrs->set(&cfg, splits);
  return cfg;
}

// CTAs that run at once in clusters of 1, 2, 4 and 8 (one an SM; a cluster
// stays within a group of SMs, so that fewer CTAs fit in large ones).
struct RowsCapacity {
  int ctas[4];
};

template <int kMode, int kBT>
RowsCapacity rows_capacity(const Operands& c) {
  static std::once_flag once[kOnceDevices];
  static RowsCapacity known[kOnceDevices];
  RowsCapacity here = {};
  auto find = [&] {
    cudaFuncSetAttribute(fp8_rows_kernel<kMode, kBT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         RowsOf<kMode, kBT>::kSmem);
    for (int i = 0; i < 4; ++i) {
      LaunchAttrs attrs;
      const cudaLaunchConfig_t cfg = rows_config<kMode, kBT>(1 << i, c.num_sms, 1, c.st, &attrs);
      int clusters = 0;
      if (cudaOccupancyMaxActiveClusters(&clusters, fp8_rows_kernel<kMode, kBT>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        clusters = i == 0 ? c.num_sms : 0;
      }
      here.ctas[i] = clusters << i;
    }
  };
  if (c.device < 0 || c.device >= kOnceDevices) {
    find();
    return here;
  }
  once_per_device(once, c.device, [&] {
    find();
    known[c.device] = here;
  });
  return known[c.device];
}

template <int kMode, int kBT>
RowsPlan plan_rows(const Operands& c, const MatmulArgs& a) {
  const RowsCapacity cap = rows_capacity<kMode, kBT>(c);
  const int64_t tiles = (a.cols + 127) / 128 * ((c.M + kBT - 1) / kBT);
  RowsPlan best = {1, INT64_MAX};
  for (int i = 0; i < 4 && (1 << i) <= a.rb; ++i) {
    const int s = 1 << i;
    if (cap.ctas[i] < s) break;
    const int64_t rounds = (tiles * s + cap.ctas[i] - 1) / cap.ctas[i];
    const int64_t blocks = (a.rb + s - 1) / s;
    int64_t cost;
    if constexpr (kMode >= kGatedForward) {
      constexpr bool kBoth = kMode == kGatedForward;             // two weights a block
      constexpr int64_t kLeast = kBoth ? (kBT <= 32 ? 43 : 60) : (kBT <= 32 ? 25 : kBT == 64 ? 31 : 48);
      constexpr int64_t kFull = kBoth ? 78 : kBT == 128 ? 52 : 39;
      constexpr int64_t kJoin[2][4] = {{40, 80, 160, 250}, {40, 100, 300, 400}};
      const int64_t busy = std::min<int64_t>(tiles * s, cap.ctas[i]);
      cost = rounds * (blocks * std::max(kLeast, kFull * busy / c.num_sms) + kJoin[kBT > 32][i]);
    } else {
      cost = rounds * (blocks * 46 + 150);
    }
    if (cost < best.cost) best = {s, cost};
  }
  return best;
}

// Tensor maps of codes [rows, cols] in boxes of box_rows x 128 bytes.
bool encode_codes(CUtensorMap* map, const uint8_t* codes, int64_t rows, int64_t cols, uint32_t box_rows) {
  const uint64_t c = static_cast<uint64_t>(cols);
  return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, c, static_cast<uint64_t>(rows), c, 128, box_rows,
                   CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int kMode, int kBT>
cudaError_t launch_rows(const Operands& c, const MatmulArgs& a) {
  const int64_t row_tiles = (a.cols + 127) / 128, m_tiles = (c.M + kBT - 1) / kBT;
  const int splits = plan_rows<kMode, kBT>(c, a).splits;
  RowsMaps<kMode> maps;
  bool ok = encode_codes(&maps.a, c.a, c.M, c.red, kBT) && encode_codes(&maps.w, c.w, c.N, c.K, 128);
  if constexpr (kMode >= kGatedForward) ok = ok && encode_codes(&maps.w2, c.w2, c.N, c.K, 128);
  if constexpr (kMode == kGatedInputGrad) ok = ok && encode_codes(&maps.a2, c.a2, c.M, c.red, kBT);
  if (!ok) return cudaErrorInvalidValue;
  LaunchAttrs attrs;
  const cudaLaunchConfig_t cfg = rows_config<kMode, kBT>(splits, row_tiles, m_tiles, c.st, &attrs);
  return cudaLaunchKernelEx(&cfg, fp8_rows_kernel<kMode, kBT>, maps, a);
}

// Columns of a pair's tile.
constexpr int64_t pair_cols(int mode) { return mode == kGatedForward ? kPairBN / 2 : kPairBN; }

template <int kMode>
cudaError_t launch_pair(const Operands& c, const MatmulArgs& args) {
  MatmulArgs a = args;
  const int64_t m_units = (c.M + 255) / 256, c_units = (a.cols + pair_cols(kMode) - 1) / pair_cols(kMode);
  if (m_units * c_units > INT32_MAX) return cudaErrorInvalidValue;
  a.m_units = static_cast<int>(m_units);
  a.units = static_cast<int>(m_units * c_units);
  PairMaps<kMode> maps;
  const uint64_t um = static_cast<uint64_t>(c.M), ucols = static_cast<uint64_t>(a.cols);
  // boxes of 32 tokens x 128 bytes (an 8-bit output: 64)
  auto encode_out = [&](CUtensorMap* map, void* out, bool bf16) {
    return encode_2d(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, out, ucols, um,
                     ucols * (bf16 ? 2 : 4), bf16 ? 64 : 32, 32, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  bool ok = encode_codes(&maps.a, c.a, c.M, c.red, 128) && encode_codes(&maps.w, c.w, c.N, c.K, 128);
  if constexpr (kMode >= kGatedForward) ok = ok && encode_codes(&maps.w2, c.w2, c.N, c.K, 128);
  if constexpr (kMode == kGatedInputGrad) ok = ok && encode_codes(&maps.a2, c.a2, c.M, c.red, 128);
  if constexpr (kMode == kGatedForward) {
    if (a.g) ok = ok && encode_out(&maps.g, a.g, true) && encode_out(&maps.u, a.u, true);
    if (a.y_scale)
      ok = ok && encode_2d(&maps.out, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.out, ucols, um, ucols, 64, 32,
                           CU_TENSOR_MAP_SWIZZLE_64B);
    else ok = ok && encode_out(&maps.out, a.out, a.out_bf16 != 0);
  } else {
    ok = ok && encode_out(&maps.out, a.out, a.out_bf16 != 0);
  }
  if (!ok) return cudaErrorInvalidValue;
  static std::once_flag once[kOnceDevices];
  once_per_device(once, c.device, [] {
    cudaFuncSetAttribute(fp8_pair_kernel<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
  });
  const int64_t pairs = std::min<int64_t>(a.units, std::max(1, c.num_sms / 2));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = c.st;
  LaunchAttrs attrs;
  attrs.set(&cfg, 2);
  return cudaLaunchKernelEx(&cfg, fp8_pair_kernel<kMode>, maps, a);
}

// Few tokens in rows, many in pairs.
template <int kMode>
cudaError_t launch_any(const Operands& c, const MatmulArgs& a) {
  // the rows kernel's tiles are grid dimensions of at most 65535; the gated
  // forward's take 64 tokens at most
  constexpr int64_t kMostTiles = 65535;
  constexpr int kMostTokens = kMode == kGatedForward ? 64 : 128;
  constexpr int64_t kPairBlock = kMode == kGatedForward ? 51 : kMode == kGatedInputGrad ? 44 : 39;
  if ((a.cols + 127) / 128 <= kMostTiles && (c.M + kMostTokens - 1) / kMostTokens <= kMostTiles) {
    if (c.M <= 16) return launch_rows<kMode, 16>(c, a);
    if (c.M <= 32) return launch_rows<kMode, 32>(c, a);
    if (c.M <= 64) return launch_rows<kMode, 64>(c, a);
    if (c.M <= kMostTokens) return launch_rows<kMode, kMostTokens>(c, a);
    // more tokens: pairs, unless their tiles leave most SMs idle for a long
    // reduction, which the rows kernel splits (512 x 3584 forward at 250
    // tokens 16.2 us on pairs, 7.8 in rows; 4096 x 4096 at 512 tokens 18.8 and
    // 20.4). Pairs: 0.39 us a block, 1 us a tile; 0.44 a block of the
    // gradient over two reductions (two of 4096 x 5504 at 256 tokens: 31.5 us on
    // pairs, 38.3 in rows); 0.51 a block of two weights (two of
    // 4112 x 3600 forward at 128 tokens: 19.0 us on pairs, 15.3 in rows; at 256 19.6
    // and 23.0; two of 11008 x 4096 at 128 37.0 and 54.3).
    const int64_t units = (c.M + 255) / 256 * ((a.cols + pair_cols(kMode) - 1) / pair_cols(kMode));
    const int64_t rounds = (units + c.num_sms / 2 - 1) / std::max(1, c.num_sms / 2);
    if (plan_rows<kMode, kMostTokens>(c, a).cost < rounds * (a.rb * kPairBlock + 100))
      return launch_rows<kMode, kMostTokens>(c, a);
  }
  return launch_pair<kMode>(c, a);
}

}  // namespace

cudaError_t launch_fp8_matmul(const Fp8Call& c) {
  const int64_t red = c.dx ? c.N : c.K, kb = (c.K + 127) / 128;
  const Operands o = {c.a, nullptr, c.w, nullptr, red, c.M, c.N, c.K, c.num_sms, c.device, c.st};
  MatmulArgs a = {};
  a.a_scale = c.a_scale;
  a.w_scale = c.w_scale;
  a.out = c.out;
  a.M = c.M;
  a.cols = c.dx ? c.K : c.N;
  a.rb = static_cast<int>((red + 127) / 128);
  a.ws_col = c.dx ? 1 : kb;
  a.ws_red = c.dx ? kb : 1;
  a.out_bf16 = c.out_bf16;
  a.accumulate = c.accumulate;
  a.mma_wait_limit = c.wait_limit;
  a.status = c.status;
  return c.dx ? launch_any<kInputGrad>(o, a) : launch_any<kForward>(o, a);
}

cudaError_t launch_gated_fwd(const GatedFwdCall& c) {
  const int64_t kb = (c.K + 127) / 128;
  const Operands o = {c.a, nullptr, c.wg, c.wu, c.K, c.M, c.N, c.K, c.num_sms, c.device, c.st};
  MatmulArgs a = {};
  a.a_scale = c.a_scale;
  a.w_scale = c.wg_scale;
  a.w_scale2 = c.wu_scale;
  a.out = c.y;
  a.M = c.M;
  a.cols = c.N;
  a.rb = static_cast<int>(kb);
  a.ws_col = kb;
  a.ws_red = 1;
  a.out_bf16 = c.y_bf16;
  a.mma_wait_limit = c.wait_limit;
  a.status = c.status;
  a.g = c.g;
  a.u = c.u;
  a.y_scale = c.y_fp8 ? c.scale : nullptr;
  a.curve = c.curve;
  return launch_any<kGatedForward>(o, a);
}

cudaError_t launch_gated_dx(const GatedDxCall& c) {
  const int64_t nb = (c.N + 127) / 128, kb = (c.K + 127) / 128;
  const Operands o = {c.dg, c.du, c.wg, c.wu, c.N, c.M, c.N, c.K, c.num_sms, c.device, c.st};
  MatmulArgs a = {};
  a.a_scale = c.dg_scale;
  a.a_scale2 = c.du_scale;
  a.w_scale = c.wg_scale;
  a.w_scale2 = c.wu_scale;
  a.out = c.out;
  a.M = c.M;
  a.cols = c.K;
  a.rb = static_cast<int>(2 * nb);
  a.rb1 = static_cast<int>(nb);
  a.ws_col = 1;
  a.ws_red = kb;
  a.out_bf16 = c.out_bf16;
  a.accumulate = c.accumulate;
  a.mma_wait_limit = c.wait_limit;
  a.status = c.status;
  return launch_any<kGatedInputGrad>(o, a);
}

}  // namespace nf4
