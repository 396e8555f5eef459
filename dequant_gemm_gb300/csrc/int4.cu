// Products of few tokens with uniform 4-bit weights in groups of 32, 64 or 128
// along a row (include/nf4gemm.h states the format):
// Y[m, n] = sum over groups of s[n, j] sum_{k in j} (q[n, k] - z[n, j]) x[m, k],
// alone or (kMats = 2) for two weights whose sums meet as act(G) U.
//
// The weight's bytes are its floor: half a byte a weight, read once for every 16
// tokens. What it takes is issue slots: a box of 16 x 256 codes costs a warp ~360
// instructions (16 tokens 540), half of them to make operands of codes, and the
// SM's four schedulers issue them at 85% of their rate while boxes go by; the first
// box is there 3 us after the launch. Measured (CUDA graph of 24 calls, weights rotated
// through more than L2, bf16, groups of 128): one token, 4096 x 4096 5.1 us, 18944 x
// 3584 9.9 us (3.6 TB/s), two of them 17.7 (4.0 TB/s); 16 tokens 12.7 and 23.2. The
// legacy mma.sync takes its operands from registers, where the codes are widened; for
// tcgen05 they would go through shared or tensor memory first, and the tensor pipe is
// 17 to 18% busy.
//
// The weight's rows are the 16 rows of mma.sync.m16n8k16, the tokens
// its 8 columns (one or two tiles). Nothing is rounded on the way: a code
// becomes the number 128 + q (bf16) or 1024 + q (fp16) by putting its four bits
// into the mantissa, the same number with the zero point is subtracted, and
// (q - z) x is exact in the fp32 sum; a group's sums are multiplied by its scale
// in fp32 and added to the row's.
//  * One CTA of 16 warps an SM, persistent: the tokens' slice of the reduction is
//    staged in shared memory once, then row tiles pass by. Of a tile, a warp has
//    16 rows and one of up to 16 parts of the slice; a cluster of up to 8 CTAs
//    splits the reduction where the rows are few or the tokens' slice is large. A
//    tile may have fewer rows than the warps could take, so that every SM has the
//    same share (3584 x 18944 at 16 tokens, 14 tiles of 16 row groups or, on 15
//    clusters, 15 of 15).
//  * A warp streams its own codes, boxes of 16 rows x 256 values, by asynchronous
//    copies into two slots of its own: no warp waits for another. A box goes into
//    registers whole (ldmatrix: word t of row g is lane (g, t)'s, which is the
//    operand's layout whatever the group), so that its slot is copied to again
//    before it is multiplied, across row tiles too.
//  * The order of k within an MMA is free as long as both operands agree. Bits of a
//    code word are taken in pairs 16 bits apart, (e1, e5), (e0, e4), (e3, e7),
//    (e2, e6) for elements e0 to e7 of 4 bytes, and the tokens are staged in that
//    order, 16 bytes a lane.
//  * Scales and zero points are loaded two boxes ahead, each by one lane of a row's
//    four, and handed to the others by shuffles, in one word (the scale's fp32 bits
//    leave the low 13 free) or two.
//  * Every warp leaves its sums of a tile in shared memory of the CTA that owns the
//    rows, which adds them in a fixed order: repeatable, no workspace.
#include <algorithm>

#include "gated.cuh"
#include "tc.cuh"

namespace nf4 {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kBoxBytes = 16 * 128;            // 16 rows x 256 codes
constexpr int kBoxCodes = 256;
constexpr int kMostSmem = 227 * 1024;
constexpr int ring_bytes(int mats) { return kWarps * 2 * kBoxBytes * mats; }
constexpr int sums_bytes(int mats, int tokens) { return kWarps * 16 * 4 * mats * tokens; }
// a box's values of a token, [word][lane], at a pitch that puts two neighbouring
// tokens, which are read together, on different banks
constexpr int kTokenBytes = kBoxCodes * 2 + 64;
constexpr int staged_bytes(int tokens) { return kTokenBytes * tokens; }

struct Int4Args {
  const uint16_t* x;             // [M, K]
  const uint8_t* codes[2];
  const uint16_t* scale[2];
  const uint8_t* zero[2];        // or null
  int64_t M, N, K;
  int groups;                    // of a row
  int boxes;                     // of a row
  int tokens, m_tiles;           // of a tile; tiles
  int shares, per_share;         // warps that stage a token; 2^16 / shares, rounded up
  int parts, per_part;           // likewise
  int splits, splits_log;
  int row_groups;                // 16 rows each, of a tile: row_groups * parts warps work
  int row_tiles, row_step;       // all; clusters that share a token tile
  int off_sums;                  // byte offset in shared memory
  bool scale_bf16, wide;
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

__device__ __forceinline__ uint4 lds_words(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

// 16 bytes from global to shared memory.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}

// d = a b, or (kAdd) d += a b
template <bool kF16>
__device__ __forceinline__ void mma_16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool add) {
  const float c[4] = {add ? d[0] : 0.0f, add ? d[1] : 0.0f, add ? d[2] : 0.0f, add ? d[3] : 0.0f};
  if constexpr (kF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t or_masked(uint32_t w, uint32_t mask, uint32_t one) {
  uint32_t v;                                  // (w & mask) | one: written out, it takes two instructions
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(v) : "r"(w), "r"(mask), "r"(one));
  return v;
}

// Codes 4 bits wide in bits 0-3 and 16-19 of w as two numbers less the zero
// point's (zz: the same two numbers made of it).
template <bool kF16>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t zz) {
  const uint32_t v = or_masked(w, 0x000f000fu, kF16 ? 0x64006400u : 0x43004300u);     // 1024, 128
  if constexpr (kF16) {
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&zz));
    return *reinterpret_cast<const uint32_t*>(&d);
  } else {
    const __nv_bfloat162 d =
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&zz));
    return *reinterpret_cast<const uint32_t*>(&d);
  }
}

// The same of bits 4-7 and 20-23 in fp16, whose mantissa has room for 1024 + 16 q:
// one exact FMA with -(64 + z) makes q - z without a shift, for a constant more a
// row and group. 8 tokens x 18944 x 3584 in groups of 128: 12.1 us for 12.8; 16 x
// 3584 x 18944 in groups of 64: 19.7 for 20.1; two weights of 18944 x 3584 at one
// token 18.9 for 20.1. Not in groups of 32 (two of 11008 x 4096 at 7 tokens: 22.5
// for 21.8) and not with two weights and two token tiles, where registers run out
// (two of 18944 x 3584 at 16: 32.0 for 31.5).
__device__ __forceinline__ uint32_t minus_64_z(uint32_t zz) {      // of twice 1024 + z
  const __half2 d = __hsub2(__float2half2_rn(960.0f), *reinterpret_cast<const __half2*>(&zz));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ uint32_t high_pair(uint32_t w, uint32_t far) {
  const uint32_t v = or_masked(w, 0x00f000f0u, 0x64006400u);
  const __half2 d = __hfma2(*reinterpret_cast<const __half2*>(&v), __float2half2_rn(0.0625f),
                            *reinterpret_cast<const __half2*>(&far));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// Sums to the shared memory of the cluster's CTA `owner` (of one: its own), at the
// address that they have in this one's.
__device__ __forceinline__ void store1(uint32_t at, uint32_t owner, bool cluster, float v) {
  if (cluster) asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(tc::mapa(at, owner)), "f"(v) : "memory");
  else asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}
__device__ __forceinline__ void store4(uint32_t at, uint32_t owner, bool cluster, float a, float b, float c, float d) {
  if (cluster)
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(tc::mapa(at, owner)), "f"(a), "f"(b),
                 "f"(c), "f"(d)
                 : "memory");
  else asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}

template <bool kF16, int kGroup, int kMats, int kNT>
__global__ void __launch_bounds__(kThreads, 1) int4_matmul_kernel(const __grid_constant__ Int4Args p) {
  constexpr int kBoxGroups = kBoxCodes / kGroup;               // 2, 4 or 8
  constexpr int kLoads = kBoxGroups / 2;                       // scales a lane loads of a box
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int parts = p.parts, row_group = warp * p.per_part >> 16, part = warp - row_group * parts;
  const int rows_tile = 16 * p.row_groups, row_warp = 16 * row_group;
  const bool works = row_warp < rows_tile;
  const int cta = static_cast<int>(blockIdx.x), rank = cta & (p.splits - 1), cluster = cta >> p.splits_log;
  const int64_t m0 = static_cast<int64_t>(cluster % p.m_tiles) * p.tokens;
  const int mt = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.M - m0));
  const int tile0 = cluster / p.m_tiles;
  // this CTA's boxes of a row, and this warp's
  const int s0 = p.boxes * rank >> p.splits_log, s1 = p.boxes * (rank + 1) >> p.splits_log;
  const int b0 = s0 + ((s1 - s0) * part * p.per_part >> 16);
  const int nb = works ? s0 + ((s1 - s0) * (part + 1) * p.per_part >> 16) - b0 : 0;
  const uint32_t ring = tc::smem_addr(smem) + warp * (2 * kMats * kBoxBytes);
  let_next_start();
  if (p.splits > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  wait_for_previous();

  // What is copied next. Box j of the warp's stream goes into slot j & 1: lane l
  // copies 16 bytes, chunk l % 8 (swizzled by the row), of rows l / 8 + 0, 4, 8
  // and 12. Of chunks and rows past the end the slot keeps what it held: any bits
  // are numbers, which meet zero scales and tokens or are dropped with their rows.
  int next_tile = tile0, next_left = 0;        // boxes left in the tile
  int64_t code_at = 0, scale_at = 0;           // this lane's first byte and scale
  int rows_left = 0, codes_left = 0;           // of this lane's rows; of the row from the box on
  const uint32_t pitch = static_cast<uint32_t>(p.K / 2);
  // lanes t = 0, 1 load the scales of row g, 2, 3 those of row g + 8, half a box's each
  const int lane_group = kLoads * (t & 1);
  const uint32_t copy_to = (lane >> 3) * 128;
  // the swizzle of rows l / 8 + 0 and + 8, and of those + 4 and + 12
  const uint32_t swizzle0 = 16 * ((lane & 7) ^ (lane >> 3)), swizzle4 = swizzle0 ^ 64;
  auto start_tile = [&] {
    next_left = next_tile < p.row_tiles ? nb : 0;
    const int64_t row0 = static_cast<int64_t>(next_tile) * rows_tile + row_warp;
    code_at = (row0 + (lane >> 3)) * pitch + static_cast<int64_t>(b0) * 128 + 16 * (lane & 7);
    rows_left = static_cast<int>(min(p.N - row0, static_cast<int64_t>(16))) - (lane >> 3);
    codes_left = static_cast<int>(p.K) - b0 * kBoxCodes;
    scale_at = min(row0 + g + 8 * (t >> 1), p.N - 1) * p.groups + b0 * kBoxGroups + lane_group;
  };
  auto copy_box = [&](uint32_t slot) {         // (address of the slot)
    if (next_left > 0) {
      const int rows = codes_left > 32 * (lane & 7) ? rows_left : 0;
#pragma unroll
      for (int mat = 0; mat < kMats; ++mat) {
        const uint8_t* src = p.codes[mat] + code_at;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * i < rows)
            copy16(slot + mat * kBoxBytes + copy_to + i * 512 + (i & 1 ? swizzle4 : swizzle0), src + i * 4 * pitch);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // a lane's kLoads scales and zero points, two scales a word and four zero points:
  // in one load each where their rows keep them aligned (p.wide)
  constexpr int kWords = (kLoads + 1) / 2;
  struct Scales {
    uint32_t s[kMats][kWords], z[kMats];
  };
  auto load_scales = [&](Scales& to) {
#pragma unroll
    for (int mat = 0; mat < kMats; ++mat) {
#pragma unroll
      for (int j = 0; j < kWords; ++j) to.s[mat][j] = 0u;
      to.z[mat] = 0x08080808u;
      if (next_left <= 0) continue;
      const uint16_t* sp = p.scale[mat] + scale_at;
      const uint8_t* zp = p.zero[mat] + scale_at;
      const int groups_left = codes_left / kGroup - lane_group;
      if (kLoads > 1 && p.wide) {              // kLoads divides the row's groups
        if (groups_left <= 0) continue;
        if constexpr (kLoads == 4) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(sp));
          to.s[mat][0] = v.x;
          to.s[mat][1] = v.y;
          if (p.zero[mat]) to.z[mat] = __ldg(reinterpret_cast<const uint32_t*>(zp));
        } else if constexpr (kLoads == 2) {
          to.s[mat][0] = __ldg(reinterpret_cast<const uint32_t*>(sp));
          if (p.zero[mat]) to.z[mat] = __ldg(reinterpret_cast<const uint16_t*>(zp));
        }
        continue;
      }
      if constexpr (kLoads == 1) {             // nothing waits for the loads here
        if (groups_left <= 0) continue;
        to.s[mat][0] = __ldg(sp);
        if (p.zero[mat]) to.z[mat] = __ldg(zp);
        continue;
      }
      uint32_t z = 0u;
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        if (j < groups_left) {
          to.s[mat][j / 2] |= static_cast<uint32_t>(__ldg(sp + j)) << (16 * (j % 2));
          if (p.zero[mat]) z |= static_cast<uint32_t>(__ldg(zp + j)) << (8 * j);
        }
      if (p.zero[mat]) to.z[mat] = z;
    }
  };
  auto advance = [&] {
    code_at += 128;
    codes_left -= kBoxCodes;
    scale_at += kBoxGroups;
    if (--next_left == 0) {
      next_tile += p.row_step;
      start_tile();
    }
  };
  // The slice's tokens, [box][token][run of 8], zeros past the ends: every warp a
  // share of one token's runs. The first box's codes are asked for before them, or
  // after the first of 16 tokens' loads, and the second's once they are here: asked
  // for at once, all SMs' boxes delay the tokens and each other (two of 18944 x 3584
  // at one token 19.3 us for 18.5, 3584 x 18944 at 16 19.5 for 18.7).
  constexpr int kFirst = kNT == 2 ? 4 : 0;
  Scales now, later;
  auto first_box = [&] {
    start_tile();
    load_scales(now);
    copy_box(ring);
    advance();
  };
  if (kFirst == 0) first_box();
  {
    // warp = share + shares tok
    const int tok = kNT == 2 ? warp : warp * p.per_share >> 16, shares = kNT == 2 ? 1 : p.shares;
    const int share = tok < p.tokens ? warp - tok * shares : shares;
    const int runs = (s1 - s0) * (kBoxCodes / 8);
    const int64_t k0 = static_cast<int64_t>(s0) * kBoxCodes;
    const int valid = tok < mt ? static_cast<int>(min(static_cast<int64_t>(runs), (p.K - k0) / 8)) : 0;
    const uint4* src = reinterpret_cast<const uint4*>(p.x + (m0 + (tok < mt ? tok : 0)) * p.K + k0);
    uint8_t* dst = smem + ring_bytes(kMats) + kTokenBytes * tok + 16 * lane;
    const int step = 32 * shares;
    auto load = [&](int r) { return r < valid ? __ldg(src + r) : make_uint4(0u, 0u, 0u, 0u); };
    auto stage = [&](int r, const uint4& v) {
      *reinterpret_cast<uint4*>(dst + (r >> 5) * (kTokenBytes * p.tokens)) =
          make_uint4(__byte_perm(v.x, v.z, 0x7632), __byte_perm(v.x, v.z, 0x5410),
                     __byte_perm(v.y, v.w, 0x7632), __byte_perm(v.y, v.w, 0x5410));
    };
    int r = share < shares ? share * 32 + lane : runs;
    uint4 first[kFirst + 1];
#pragma unroll
    for (int i = 0; i < kFirst; ++i) first[i] = load(r + i * step);
    if (kFirst > 0) first_box();
#pragma unroll
    for (int i = 0; i < kFirst; ++i, r += step)
      if (r < runs) stage(r, first[i]);
#pragma unroll 4
    for (; r < runs; r += step) stage(r, load(r));
  }
  load_scales(later);
  copy_box(ring + kMats * kBoxBytes);
  advance();
  __syncthreads();

  // of each 16 rows, CTA r of the cluster owns the run of 16 / splits from r 16 / splits
  const int own = rows_tile >> p.splits_log, run_log = 4 - p.splits_log, run = 1 << run_log;
  const uint32_t inbox = tc::smem_addr(smem) + p.off_sums;
  // lanes 8 j .. 8 j + 7 give the rows of matrix j, chunk 4 c + j of a box's rows
  const uint32_t lm = (lane & 7) * 128 + 16 * ((lane >> 3) ^ (lane & 7));
  // A lane whose column of the MMA has no token reads another's: the column's sums
  // are dropped.
  const uint32_t x_box = kTokenBytes * p.tokens;
  const uint32_t x_first = tc::smem_addr(smem) + ring_bytes(kMats) + kTokenBytes * (g < p.tokens ? g : 0) + 16 * t +
                           (b0 - s0) * x_box;
  uint32_t slot = ring;
  for (int tile = tile0; tile < p.row_tiles; tile += p.row_step) {
    float acc[kMats][kNT][4] = {};
    uint32_t xb = x_first;
#pragma unroll 1
    for (int b = 0; b < nb; ++b, xb += x_box) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();
      uint32_t q[kMats][2][2][4];              // [weight][chunk][row half][word]
#pragma unroll
      for (int mat = 0; mat < kMats; ++mat)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            ldmatrix4(slot + mat * kBoxBytes + h * 1024 + (c ? lm ^ 64u : lm), q[mat][c][h]);
      // this box's scales as fp32 bits, and twice 128 + z or 1024 + z (a code's numbers
      // less q); in groups of 32, where registers run out, z in the scale's low bits.
      // Apart against together: two of 18944 x 3584 at one token 18.2 us for 18.4, at
      // 16 23.9 for 24.2; groups of 32, two of 11008 x 4096 at 7 22.2 for 21.6.
      constexpr uint32_t kOne = kF16 ? 0x64u : 0x43u;
      constexpr bool kApart = kGroup > 32;
      uint32_t sz[kMats][kLoads], zz[kMats][kLoads];
#pragma unroll
      for (int mat = 0; mat < kMats; ++mat)
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          const uint32_t bits = now.s[mat][j / 2] >> (16 * (j % 2)) & 0xffffu;
          sz[mat][j] = __float_as_uint(scale_value(bits, p.scale_bf16));
          if (kApart) zz[mat][j] = __byte_perm(now.z[mat], kOne, 0x4040 + 0x0101 * j);
          else sz[mat][j] |= now.z[mat] >> (8 * j) & 0xffu;
        }
      __syncwarp();
      now = later;
      load_scales(later);
      copy_box(slot);
      advance();
      slot = 2 * ring + kMats * kBoxBytes - slot;              // the other one
#pragma unroll
      for (int j = 0; j < kBoxGroups; ++j) {
        constexpr bool kHigh = kF16 && kGroup > 32 && kMats * kNT < 4;
        uint32_t za[kMats], zb[kMats], far_a[kMats], far_b[kMats];
        float sa[kMats], sb[kMats];
#pragma unroll
        for (int mat = 0; mat < kMats; ++mat) {
          const int from = (lane & 28) + j / kLoads;
          const uint32_t va = __shfl_sync(0xffffffffu, sz[mat][j % kLoads], from);
          const uint32_t vb = __shfl_sync(0xffffffffu, sz[mat][j % kLoads], from + 2);
          za[mat] = kApart ? __shfl_sync(0xffffffffu, zz[mat][j % kLoads], from) : __byte_perm(va, kOne, 0x4040);
          zb[mat] = kApart ? __shfl_sync(0xffffffffu, zz[mat][j % kLoads], from + 2) : __byte_perm(vb, kOne, 0x4040);
          far_a[mat] = kHigh ? minus_64_z(za[mat]) : 0u;
          far_b[mat] = kHigh ? minus_64_z(zb[mat]) : 0u;
          sa[mat] = __uint_as_float(kApart ? va : va & 0xffffff00u);
          sb[mat] = __uint_as_float(kApart ? vb : vb & 0xffffff00u);
        }
        float sum[kMats][kNT][4];
#pragma unroll
        for (int i = 0; i < 8 / kBoxGroups; ++i) {
          const int w = j * (8 / kBoxGroups) + i;              // of the box's 8 words a lane
          uint4 x[kNT];
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) x[nt] = lds_words(xb + 64 * w + 8 * kTokenBytes * nt);
#pragma unroll
          for (int mat = 0; mat < kMats; ++mat) {
            const uint32_t wa = q[mat][w >> 2][0][w & 3], wb = q[mat][w >> 2][1][w & 3];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t a[4] = {code_pair<kF16>(wa >> (8 * h), za[mat]), code_pair<kF16>(wb >> (8 * h), zb[mat]),
                                     kHigh ? high_pair(wa >> (8 * h), far_a[mat])
                                           : code_pair<kF16>(wa >> (8 * h + 4), za[mat]),
                                     kHigh ? high_pair(wb >> (8 * h), far_b[mat])
                                           : code_pair<kF16>(wb >> (8 * h + 4), zb[mat])};
#pragma unroll
              for (int nt = 0; nt < kNT; ++nt)
                mma_16<kF16>(sum[mat][nt], a, h ? x[nt].z : x[nt].x, h ? x[nt].w : x[nt].y, i + h > 0);
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
    }

    // every warp's sums to the CTA that owns the rows: [split, part][weight][token][row],
    // or with 16 tokens [split, part][weight][row][token], where a lane's four of a row
    // (tokens 2 t, 2 t + 1, 8 more) are one store and one load, swizzled so that eight
    // rows' are on different banks (sum by sum, two of 18944 x 3584 at 16 tokens took
    // 29.2 us for 23.8).
    // The first wait: every CTA runs, and has read its last tile's sums. (A CTA by
    // itself uses its own barrier: with cluster barriers a tile took 2 us more.)
    if (p.splits > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    else if (tile != tile0) __syncthreads();
    const int from = (rank * parts + part) * kMats;
#pragma unroll
    for (int mat = 0; mat < kMats; ++mat)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = row_warp + g + 8 * (e >> 1), local = (row >> 4 << run_log) + (row & (run - 1));
        const uint32_t owner = (row & 15) >> run_log;
        if (!works) continue;
        if constexpr (kNT == 2) {
          if (e & 1) continue;
          const uint32_t at = inbox + 16u * (((from + mat) * own + local) * 4 + (t ^ (local >> 1 & 3)));
          const float *lo = acc[mat][0] + e, *hi = acc[mat][kNT - 1] + e;
          store4(at, owner, p.splits > 1, lo[0], lo[1], hi[0], hi[1]);
        } else {
          const int tok = 2 * t + (e & 1);
          if (tok >= mt) continue;
          store1(inbox + 4u * (((from + mat) * mt + tok) * own + local), owner, p.splits > 1, acc[mat][0][e]);
        }
      }
    if (p.splits > 1) tc::cluster_sync();
    else __syncthreads();
    const float* sums = reinterpret_cast<const float*>(smem + p.off_sums);
    constexpr int kEach = kNT == 2 ? 4 : 1;    // tokens a thread adds up at once
    const int items = kNT == 2 ? 4 * own : mt * own;
    for (int i = threadIdx.x; i < items; i += kThreads) {
      const int col = kNT == 2 ? (i >= own) + (i >= 2 * own) + (i >= 3 * own) : mt == 1 ? 0 : i / own;
      const int row = i - col * own;
      const int64_t n = static_cast<int64_t>(tile) * rows_tile + ((row >> run_log) << 4) + (rank << run_log) +
                        (row & (run - 1));
      if (n >= p.N) continue;
      float y[kMats][kEach] = {};
#pragma unroll 4
      for (int k = 0; k < p.splits * parts; ++k)
#pragma unroll
        for (int mat = 0; mat < kMats; ++mat) {
          if constexpr (kNT == 2) {
            const float4 v =
                reinterpret_cast<const float4*>(sums)[((k * kMats + mat) * own + row) * 4 + (col ^ (row >> 1 & 3))];
            y[mat][0] += v.x;
            y[mat][1] += v.y;
            y[mat][2] += v.z;
            y[mat][3] += v.w;
          } else {
            y[mat][0] += sums[((k * kMats + mat) * mt + col) * own + row];
          }
        }
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const int tok = kNT == 2 ? 2 * col + (e & 1) + 8 * (e >> 1) : col;
        if (tok >= mt) continue;
        const float v = kMats == 2 ? gated(y[0][e], y[kMats - 1][e], p.curve) : y[0][e];
        store_sum(p.y, p.y_elem, (m0 + tok) * p.N + n, v, p.accumulate);
      }
    }
    if (p.splits > 1 && tile + p.row_step < p.row_tiles)
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Launch shape of a call: tokens of a tile, parts of a slice, splits (the cluster),
// row groups of a tile and clusters for each token tile. Estimated time, in us: a
// box a warp takes 1.15 us and weight where all 16 warps work (1.2 above 8 tokens),
// less where fewer do, as the issue slots of the SM's four schedulers bound it, down
// to 0.55 of it; a tile 1 us more for its sums, 0.015 a token and weight, 0.01 a part,
// 0.05 to 0.15 in clusters of 2 to 8; staging 50 bytes a ns. Fitted to every shape of
// 136 calls (1 to 32 tokens, 512 x 3584 to 18944 x 3584, alone and gated), of which
// it takes one within 1.2% of the fastest on average, 11% at worst: 11008 x 4096 at
// one token 8.4 us in three parts (8.9 in two), 4096 x 11008 8.8 in rows of a CTA (9.1
// in clusters of 2), 3584 x 18944 at 16 tokens 16.1 in clusters of 8 (21.7 of 4).
struct Int4Shape {
  int tokens, parts, splits_log, row_groups;
  int row_tiles, row_step, m_tiles;
};

Int4Shape plan_int4(int64_t M, int64_t N, int boxes, int mats, const int (&ctas)[4]) {
  Int4Shape best = {};
  float best_cost = 3e38f;
  const int groups = static_cast<int>((N + 15) / 16);
  for (int tokens = 16; tokens >= 1; tokens /= 2) {
    if (tokens > 1 && tokens / 2 >= M) continue;            // a smaller tile holds them all
    const int mt = M >= tokens || tokens == 16 ? tokens : static_cast<int>(M);   // two column tiles hold 16
    const int room = (kMostSmem - ring_bytes(mats) - sums_bytes(mats, mt)) / staged_bytes(mt);
    const int m_tiles = static_cast<int>((M + mt - 1) / mt);
    const float box = (mt > 8 ? 1.2f : 1.15f) * static_cast<float>(mats);
    for (int sl = 0; sl < 4 && (1 << sl) <= boxes; ++sl) {
      const int slice = (boxes + (1 << sl) - 1) >> sl, clusters = ctas[sl] >> sl;
      if (slice > room || clusters == 0) continue;
      const int step = std::max(1, clusters / m_tiles);
      const float staged = static_cast<float>(slice) * static_cast<float>(staged_bytes(mt));
      const float fixed = staged / 50000.0f + (sl > 0 ? 1.3f : 0.9f);
      const float sums = 1.0f + 0.015f * static_cast<float>(mt * mats) + 0.05f * static_cast<float>(sl);
      for (const int parts : {1, 2, 3, 4, 5, 8, 16}) {
        // the passes that full tiles take, then the smallest tile that takes no more
        const int full = kWarps / parts, tiles = (groups + full - 1) / full, passes = (tiles + step - 1) / step;
        const int spread = passes * step;
        const int rg = groups <= spread ? 1 : (groups - 1) / spread + 1;
        const int row_tiles = (groups + rg - 1) / rg, row_step = std::min(row_tiles, step);
        const int64_t all = static_cast<int64_t>(row_step) * m_tiles;
        const float waves = static_cast<float>((all + clusters - 1) / clusters);
        // of the fullest of four schedulers
        const float busy = std::max(0.55f, static_cast<float>((rg * parts + 3) / 4) / 4.0f);
        const float each = std::max(1.0f, static_cast<float>(slice) / static_cast<float>(parts));
        const float tile = each * box * busy + sums + 0.01f * static_cast<float>(parts << sl);
        const float cost = waves * (static_cast<float>(passes) * tile + fixed);
        if (cost < best_cost) {
          best_cost = cost;
          best = {mt, parts, sl, rg, row_tiles, row_step, m_tiles};
        }
      }
    }
    if (best_cost < 3e38f) break;                           // fewer tokens read the weight more often
  }
  return best;
}

template <bool kF16, int kGroup, int kMats, int kNT>
cudaError_t launch_int4_as(const Int4Call& c, const Int4Shape& shape) {
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
  a.boxes = static_cast<int>((a.K + kBoxCodes - 1) / kBoxCodes);
  a.tokens = shape.tokens;
  a.m_tiles = shape.m_tiles;
  a.shares = kWarps / shape.tokens;
  a.per_share = (65536 + a.shares - 1) / a.shares;
  a.parts = shape.parts;
  a.per_part = (65536 + a.parts - 1) / a.parts;
  a.splits = 1 << shape.splits_log;
  a.splits_log = shape.splits_log;
  a.row_groups = shape.row_groups;
  a.row_tiles = shape.row_tiles;
  a.row_step = shape.row_step;
  const int slice = (a.boxes + a.splits - 1) / a.splits;
  a.off_sums = ring_bytes(kMats) + slice * staged_bytes(shape.tokens);
  a.scale_bf16 = c.w[0].scale_elem == kElemBf16;
  // a lane's scales and zero points in one load each
  constexpr uint32_t kLoads = 128 / kGroup;
  a.wide = a.groups % kLoads == 0;
  for (int i = 0; i < kMats; ++i)
    a.wide = a.wide && reinterpret_cast<uintptr_t>(a.scale[i]) % (2 * kLoads) == 0 &&
             reinterpret_cast<uintptr_t>(a.zero[i]) % kLoads == 0;
  a.curve = c.curve;
  a.y = c.y;
  a.y_elem = c.y_elem;
  a.accumulate = c.accumulate;
  static std::once_flag once[kOnceDevices];
  once_per_device(once, c.device, [] {
    cudaFuncSetAttribute(int4_matmul_kernel<kF16, kGroup, kMats, kNT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         kMostSmem);
  });
  const int64_t grid = static_cast<int64_t>(shape.row_step) * shape.m_tiles * a.splits;
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(a.off_sums) + sums_bytes(kMats, shape.tokens);
  cfg.stream = c.st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(a.splits);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, int4_matmul_kernel<kF16, kGroup, kMats, kNT>, a);
}

// CTAs that run at once in clusters of 1, 2, 4 and 8, one an SM (a cluster stays
// within a group of SMs); the same for every kernel above.
struct Int4Capacity {
  int ctas[4];
};

Int4Capacity int4_capacity(const Int4Call& c) {
  static std::once_flag once[kOnceDevices];
  static Int4Capacity known[kOnceDevices];
  Int4Capacity here = {};
  auto find = [&] {
    auto kernel = int4_matmul_kernel<false, 128, 1, 2>;
    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
    for (int i = 0; i < 4; ++i) {
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 1u << i;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(c.num_sms) << i);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = kMostSmem;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int clusters = 0;
      if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess) {
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

template <typename F>
cudaError_t with_group(int group, F&& go) {
  if (group == 32) return go(std::integral_constant<int, 32>{});
  if (group == 64) return go(std::integral_constant<int, 64>{});
  return go(std::integral_constant<int, 128>{});
}

}  // namespace

cudaError_t launch_int4_matmul(const Int4Call& c) {
  const Int4Shape shape = plan_int4(c.M, c.w[0].rows, static_cast<int>((c.w[0].cols + kBoxCodes - 1) / kBoxCodes),
                                    c.gated ? 2 : 1, int4_capacity(c).ctas);
  if (shape.row_groups == 0) return cudaErrorInvalidConfiguration;
  return with_group(c.w[0].group, [&](auto g) {
    constexpr int kGroup = decltype(g)::value;
    auto go = [&](auto f16, auto mats) {
      constexpr bool kF16 = decltype(f16)::value;
      constexpr int kMats = decltype(mats)::value;
      return shape.tokens <= 8 ? launch_int4_as<kF16, kGroup, kMats, 1>(c, shape)
                               : launch_int4_as<kF16, kGroup, kMats, 2>(c, shape);
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
