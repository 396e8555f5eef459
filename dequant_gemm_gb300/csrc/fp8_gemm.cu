// Products of block-scaled e4m3 operands (fp8.cuh):
//   forward    Y[m, n]  = sum_b sx[m, b] sw[n / 128, b] sum_{k in b} qx[m, k] qw[n, k]
//   input grad dX[m, k] = sum_b sy[m, b] sw[b, k / 128] sum_{n in b} qy[m, n] qw[n, k]
// (b: the 128-wide blocks of the reduction; the weight is frozen, so there is
// no weight gradient.)
//
// The inner sums run on the tensor cores (tcgen05, kind::f8f6f4, fp32
// accumulators in tensor memory). The scales are fp32 and differ from block
// to block along the reduction, so no accumulator can run on across blocks:
// each block's sums go to a fresh tensor-memory buffer, and warps read them
// back, multiply by the block's scales and add them into fp32 totals held in
// registers, while the tensor cores fill the next buffer.
#include <algorithm>

#include "fp8.cuh"
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
constexpr int kPairOffBars = kPairOffScale + 2 * kScaleBytes;
constexpr int kPairSmem = kPairOffBars + 256 + 1024;   // + alignment slack
static_assert(kPairSmem <= 227 * 1024, "shared memory");

template <bool kDx>
__global__ void __launch_bounds__(kPairThreads, 1)
fp8_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                const __grid_constant__ CUtensorMap tm_out, const MatmulArgs p) {
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
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kPairOffBars + 8 * (2 * kPairStages + 9));
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
    *abort_flag = 0;
    tc::fence_barrier_init();
    tc::prefetch_tensormap(&tm_a);
    tc::prefetch_tensormap(&tm_w);
    tc::prefetch_tensormap(&tm_out);
  }
  if (warp == 1) tc::tmem_alloc<2>(tc::smem_addr(tmem_slot), 512);
  tc::fence_before_sync();
  tc::cluster_sync();                  // the peer's barriers exist before any arrival
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  let_next_start();
  wait_for_previous();

  auto fail = [&](uint32_t role) {
    report_status(p.status, kStatusTimeout, kDx ? kSiteFp8Dx : kSiteFp8Fwd, role);
    *abort_flag = 1;
    const uint32_t peer = tc::mapa(tc::smem_addr(const_cast<int*>(abort_flag)), rank ^ 1u);
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer), "r"(1u) : "memory");
  };
  auto tile_m = [&](int u) { return static_cast<int64_t>(u % p.m_units) * 256 + rank * 128; };
  const int64_t col_blocks = (p.cols + 127) / 128;
  auto tile_c = [&](int u) { return static_cast<int64_t>(u / p.m_units) * kPairBN; };

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
        const int32_t c = static_cast<int32_t>(tile_c(u)) + static_cast<int32_t>(rank) * 128;
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
            tc::mbar_arrive_expect_tx(full_bar(slot), kPairStageBytes);
            tc::tma_load_2d(dst, &tm_a, i * 128, m, full_bar(slot));
            if (kDx) tc::tma_load_2d(dst + kTileBytes, &tm_w, c, i * 128, full_bar(slot));
            else tc::tma_load_2d(dst + kTileBytes, &tm_w, i * 128, c, full_bar(slot));
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
        const int64_t m0 = tile_m(u), cb = tile_c(u) / 128 + (lane >> 4);
        const int tokens = static_cast<int>(min(p.M - m0, static_cast<int64_t>(128)));
        const float* src = p.a_scale + (m0 + t0) * p.rb + j;
        const float* wsrc = p.w_scale + cb * p.ws_col + j * p.ws_red;
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
#pragma unroll 2
          for (int t = t0; t < 128; t += 4)
            copy4(dst + 4 * t, src + i + static_cast<int64_t>(t < n ? t - t0 : 0) * p.rb, t < n);
          if (warp == 2) copy4(dst + 4 * (128 + (lane >> 4)), wsrc + i * p.ws_red, n > 0 && w_in);
          arrive_on_copies(sfull_bar(ch & 1));
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");   // also after an abort
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPairManyRegs));
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t src = tmem + (static_cast<uint32_t>(32 * q) << 16) + 128u * half;
    const uint32_t box_addr = base + kPairOffBox + (warp - 4) * 2 * kBoxBytes;
    const int row = 32 * q + lane;       // token of this thread within the CTA's 128
    const uint32_t scales = base + kPairOffScale;

    int ch = 0;
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
        const float sa = lds(sp + 4 * row), sw = lds(sp + 4 * (128 + half));
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
        const float s = sa * sw;
        if (in == kScaleChunk - 1 || i + 1 == p.rb) {
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(sempty_bar(ch & 1));
          ++ch;
        }
        tc::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 4; ++k) scale_add(acc + 16 * k, v[k], s);
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld16f(src + 256u * b + 64u + 16u * k, v[k]);
        tc::tmem_wait_ld();
        tc::fence_before_sync();         // all read: the buffer is free
        if (lane == 0) arrive_relaxed(read_remote + 8u * b);
#pragma unroll
        for (int k = 0; k < 4; ++k) scale_add(acc + 64 + 16 * k, v[k], s);
        b ^= 1u;
        sum_ph ^= b ^ 1u;
      }
      if (stop) break;
      // out: 128 columns of 32 tokens a warp, in boxes of 128 bytes a row whose
      // 16-byte chunks are swizzled by the row (no bank conflicts); rows and
      // columns past the end are dropped by the copy
      const int64_t m0 = tile_m(u) + 32 * q, m = m0 + lane, c0 = tile_c(u) + 128 * half;
      if (m0 >= p.M || c0 >= p.cols) continue;
      if (p.accumulate && m < p.M) {
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
      auto send = [&](int64_t c, int k) {
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0 && c < p.cols) {
          tc::tma_store_2d(&tm_out, box_addr + (k & 1) * kBoxBytes, static_cast<int32_t>(c), static_cast<int32_t>(m0));
          tc::bulk_commit();
        }
      };
      auto reuse = [&] {                 // the box's previous contents have been read
        if (lane == 0) tc::bulk_wait_read_all();
        __syncwarp();
      };
      const uint32_t rowp = box_addr + 128 * lane;
      if (p.out_bf16) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 0) reuse();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float* a = acc + 64 * h + 8 * j;
            sts128(rowp + h * kBoxBytes + 16 * (j ^ (lane & 7)), pack2<kElemBf16>(a[0], a[1]), pack2<kElemBf16>(a[2], a[3]),
                   pack2<kElemBf16>(a[4], a[5]), pack2<kElemBf16>(a[6], a[7]));
          }
          send(c0 + 64 * h, h);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          if (h % 2 == 0) reuse();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float* a = acc + 32 * h + 4 * j;
            sts128(rowp + (h & 1) * kBoxBytes + 16 * (j ^ (lane & 7)), __float_as_uint(a[0]), __float_as_uint(a[1]),
                   __float_as_uint(a[2]), __float_as_uint(a[3]));
          }
          send(c0 + 32 * h, h);
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
template <int kBT>
struct RowsCfg {
  static constexpr int kGroups = kBT >= 64 ? 2 : 1;      // token groups, four warps each
  static constexpr int kCols = kBT / kGroups;            // tokens a thread
  static constexpr int kTotalWarps = 4 * kGroups;
  static constexpr int kThreads = 32 * (4 + kTotalWarps);
  static constexpr int kStageBytes = kTileBytes + kBT * 128;
  // what fits beside the inbox: 7 to 10 weight tiles of 16 KB in flight up to 64
  // tokens, 4 at 128, above the 35 KB an SM needs to keep HBM busy
  static constexpr int kStages = kBT == 128 ? 4 : kBT == 64 ? 7 : kBT == 32 ? 8 : 10;
  static constexpr int kBufs = kBT == 128 ? 4 : 8;
  static constexpr int kTmemCols = kBufs * kBT;          // 128, 256, 512, 512
  static constexpr int kPitch = kBT + 4;                 // scale row: 16-byte aligned
  static constexpr int kChunkBytes = kScaleChunk * kPitch * 4;
  static constexpr int kOffInbox = kStages * kStageBytes;
  static constexpr int kOffScale = kOffInbox + kBT * 512;
  static constexpr int kOffBars = kOffScale + 2 * kChunkBytes;
  static constexpr int kNumBars = 2 * kStages + 2 * kBufs + 4 + 1;
  static constexpr int kSmem = kOffBars + 8 * kNumBars + 16 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kTmemCols <= 512, "tensor memory");
};

template <bool kDx, int kBT>
__global__ void __launch_bounds__(RowsCfg<kBT>::kThreads, 1)
fp8_rows_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                const MatmulArgs p) {
  using C = RowsCfg<kBT>;
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
    tc::prefetch_tensormap(&tm_a);
    tc::prefetch_tensormap(&tm_w);
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
    report_status(p.status, kStatusTimeout, kDx ? kSiteFp8Dx : kSiteFp8Fwd, role);
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
      const int32_t k = (b0 + i) * 128;
      if (tc::elect_one()) {
        tc::mbar_arrive_expect_tx(full_bar(slot), C::kStageBytes);
        if (kDx) tc::tma_load_2d(dst, &tm_w, static_cast<int32_t>(r0), k, full_bar(slot));
        else tc::tma_load_2d(dst, &tm_w, k, static_cast<int32_t>(r0), full_bar(slot));
        tc::tma_load_2d(dst + kTileBytes, &tm_a, k, static_cast<int32_t>(m0), full_bar(slot));
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
    const uint64_t bdesc0 = tc::sw128_kmajor_desc(base + kTileBytes);
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
        for (int j = 0; j < 4; ++j)
          mma_f8_ss<1>(tmem + buf * kBT, adesc0 + off + kAStep * j, bdesc0 + off + 2u * j, idesc,
                       j != 0 ? 1u : 0u);
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
    const float* as = p.a_scale + (m0 + t0) * p.rb + b0 + j;
    const float* ws = p.w_scale + (r0 / 128) * p.ws_col + (b0 + j) * p.ws_red;
    for (int i = 0, ch = 0; i < nb; i += kScaleChunk, ++ch) {
      if (!waited(sempty_bar(ch & 1), ((ch >> 1) & 1) ^ 1, kRoleProducer)) break;
      const uint32_t dst = base + C::kOffScale + (ch & 1) * C::kChunkBytes + j * (C::kPitch * 4);
      const int n = i + j < nb ? tokens : 0;
#pragma unroll 8
      for (int t = t0; t < kBT; t += 4)
        copy4(dst + 4 * t, as + i + static_cast<int64_t>(t < n ? t - t0 : 0) * p.rb, t < n);
      if (warp == 2 && lane < 16) copy4(dst + 4 * kBT, ws + i * p.ws_red, n > 0);
      arrive_on_copies(sfull_bar(ch & 1));
    }
    asm volatile("cp.async.wait_all;" ::: "memory");   // also after an abort
  } else {
    const int q = warp & 3, part = (warp - 4) >> 2;
    const uint32_t src = tmem + (static_cast<uint32_t>(32 * q) << 16) + C::kCols * part;
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
      const float w = lds(sp + 4 * kBT);
#pragma unroll
      for (int c = 0; c < C::kCols; c += 16) {
        float v[16];
        tmem_ld16f(src + kBT * buf + c, v);
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
    const int part = (warp - 4) >> 2, col = 32 * (warp & 3) + lane;
#pragma unroll
    for (int j = 0; j < C::kCols; ++j) {
      const int t = C::kCols * part + j;
      const uint32_t at = base + C::kOffInbox + 4u * ((rank * own + (t & (own - 1))) * 128 + col);
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
    if (m >= p.M || r0 + c >= p.cols) continue;
    const uint32_t at = base + C::kOffInbox + 4u * (t * 128 + c);
    float4 y = lds128(at);
    for (int k = 1; k < splits; ++k) {
      const float4 z = lds128(at + 512u * own * k);
      y.x += z.x;
      y.y += z.y;
      y.z += z.z;
      y.w += z.w;
    }
    const int64_t o = m * p.cols + r0 + c;
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
struct RowsPlan {
  int splits;
  int64_t cost;
};

template <bool kDx, int kBT>
cudaLaunchConfig_t rows_config(int splits, int64_t row_tiles, int64_t m_tiles, cudaStream_t st,
                               LaunchAttrs* attrs) {
  using C = RowsCfg<kBT>;
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

template <bool kDx, int kBT>
RowsCapacity rows_capacity(const Fp8Call& c) {
  static std::once_flag once[kOnceDevices];
  static RowsCapacity known[kOnceDevices];
  RowsCapacity here = {};
  auto find = [&] {
    cudaFuncSetAttribute(fp8_rows_kernel<kDx, kBT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         RowsCfg<kBT>::kSmem);
    for (int i = 0; i < 4; ++i) {
      LaunchAttrs attrs;
      const cudaLaunchConfig_t cfg = rows_config<kDx, kBT>(1 << i, c.num_sms, 1, c.st, &attrs);
      int clusters = 0;
      if (cudaOccupancyMaxActiveClusters(&clusters, fp8_rows_kernel<kDx, kBT>, &cfg) != cudaSuccess) {
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

template <bool kDx, int kBT>
RowsPlan plan_rows(const Fp8Call& c, const MatmulArgs& a) {
  const RowsCapacity cap = rows_capacity<kDx, kBT>(c);
  const int64_t tiles = (a.cols + 127) / 128 * ((c.M + kBT - 1) / kBT);
  RowsPlan best = {1, INT64_MAX};
  for (int i = 0; i < 4 && (1 << i) <= a.rb; ++i) {
    const int s = 1 << i;
    if (cap.ctas[i] < s) break;
    const int64_t rounds = (tiles * s + cap.ctas[i] - 1) / cap.ctas[i];
    const int64_t cost = rounds * ((a.rb + s - 1) / s * 46 + 150);
    if (cost < best.cost) best = {s, cost};
  }
  return best;
}

template <bool kDx, int kBT>
cudaError_t launch_rows(const Fp8Call& c, const MatmulArgs& a, int64_t red) {
  const int64_t row_tiles = (a.cols + 127) / 128, m_tiles = (c.M + kBT - 1) / kBT;
  const int splits = plan_rows<kDx, kBT>(c, a).splits;
  CUtensorMap tm_a, tm_w;
  const uint64_t ur = static_cast<uint64_t>(red), um = static_cast<uint64_t>(c.M);
  if (!encode_2d(&tm_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.a, ur, um, ur, 128, kBT,
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.w, static_cast<uint64_t>(c.K),
                 static_cast<uint64_t>(c.N), static_cast<uint64_t>(c.K), 128, 128,
                 CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  LaunchAttrs attrs;
  const cudaLaunchConfig_t cfg = rows_config<kDx, kBT>(splits, row_tiles, m_tiles, c.st, &attrs);
  return cudaLaunchKernelEx(&cfg, fp8_rows_kernel<kDx, kBT>, tm_a, tm_w, a);
}

template <bool kDx>
cudaError_t launch_pair(const Fp8Call& c, const MatmulArgs& args, int64_t red) {
  MatmulArgs a = args;
  const int64_t m_units = (c.M + 255) / 256, c_units = (a.cols + kPairBN - 1) / kPairBN;
  a.m_units = static_cast<int>(m_units);
  a.units = static_cast<int>(m_units * c_units);
  CUtensorMap tm_a, tm_w, tm_out;
  const uint64_t ur = static_cast<uint64_t>(red), um = static_cast<uint64_t>(c.M);
  const uint64_t pitch = static_cast<uint64_t>(a.cols) * (c.out_bf16 ? 2 : 4);
  if (!encode_2d(&tm_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.a, ur, um, ur, 128, 128,
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.w, static_cast<uint64_t>(c.K),
                 static_cast<uint64_t>(c.N), static_cast<uint64_t>(c.K), 128, 128,
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&tm_out, c.out_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                 c.out, static_cast<uint64_t>(a.cols), um, pitch, c.out_bf16 ? 64 : 32, 32,
                 CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  static std::once_flag once[kOnceDevices];
  once_per_device(once, c.device, [] {
    cudaFuncSetAttribute(fp8_pair_kernel<kDx>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
  });
  const int64_t pairs = std::min<int64_t>(a.units, std::max(1, c.num_sms / 2));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = c.st;
  LaunchAttrs attrs;
  attrs.set(&cfg, 2);
  return cudaLaunchKernelEx(&cfg, fp8_pair_kernel<kDx>, tm_a, tm_w, tm_out, a);
}

template <bool kDx>
cudaError_t launch_any(const Fp8Call& c) {
  const int64_t red = kDx ? c.N : c.K, kb = (c.K + 127) / 128;
  MatmulArgs a = {};
  a.a_scale = c.a_scale;
  a.w_scale = c.w_scale;
  a.out = c.out;
  a.M = c.M;
  a.cols = kDx ? c.K : c.N;
  a.rb = static_cast<int>((red + 127) / 128);
  a.ws_col = kDx ? 1 : kb;
  a.ws_red = kDx ? kb : 1;
  a.out_bf16 = c.out_bf16;
  a.accumulate = c.accumulate;
  a.mma_wait_limit = c.wait_limit;
  a.status = c.status;
  // the rows kernel's tiles are grid dimensions of at most 65535
  constexpr int64_t kMostTiles = 65535;
  if ((a.cols + 127) / 128 <= kMostTiles && (c.M + 127) / 128 <= kMostTiles) {
    if (c.M <= 16) return launch_rows<kDx, 16>(c, a, red);
    if (c.M <= 32) return launch_rows<kDx, 32>(c, a, red);
    if (c.M <= 64) return launch_rows<kDx, 64>(c, a, red);
    if (c.M <= 128) return launch_rows<kDx, 128>(c, a, red);
    // more tokens: pairs, unless their tiles leave most SMs idle for a long
    // reduction, which the rows kernel splits (512 x 3584 forward at 250
    // tokens 16.2 us on pairs, 7.8 in rows; 4096 x 4096 at 512 tokens 18.8 and
    // 20.4). Pairs: 0.39 us a block, 1 us a tile.
    const int64_t units = (c.M + 255) / 256 * ((a.cols + kPairBN - 1) / kPairBN);
    const int64_t rounds = (units + c.num_sms / 2 - 1) / std::max(1, c.num_sms / 2);
    if (plan_rows<kDx, 128>(c, a).cost < rounds * (a.rb * 39 + 100)) return launch_rows<kDx, 128>(c, a, red);
  }
  return launch_pair<kDx>(c, a, red);
}

}  // namespace

cudaError_t launch_fp8_matmul(const Fp8Call& c) { return c.dx ? launch_any<true>(c) : launch_any<false>(c); }

}  // namespace nf4
