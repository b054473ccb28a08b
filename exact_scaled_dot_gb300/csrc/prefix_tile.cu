// prefix_tile.cu -- the keys that a whole batch shares, for the query rows of
// all its sequences: the first part of attn_fwd_prefix_cache (prefix_cache.cu) where
// there are enough rows for the tensor core's 128-row tiles, on sm_103a.
//
// With rows = (sequences) x (query heads of a KV head) x n_q the prefix costs
// 2 rows (d_h + d_v) operations per key and head for 0.5625 (d_h + d_v) bytes:
// from a few hundred rows on it is bound by the tensor core, not by memory.  A
// CTA takes a range of the prefix for one KV head and up to 256 rows, and turns
// every tile of 64 keys (two pages) into fp16 operands once for all of them.
//
// Scores.  With q = Q's row times a power of two and k = s (c - z) per group of
// 64 dims, q . k = sum_g [ q_g . s_g (c - 8)_g + (sum q_g) s_g (8 - z_g) ].  s has
// 8 significant bits and |c - 8| <= 8, so that s (c - 8) is exact in fp16 (times a
// power of two 2^e of the tile; s (c - z) would need a bit more).  The second
// term is one more step of the product's inner dimension, with sum q_g as three
// fp16 numbers (33 bits).  So the scores are exact products summed in fp32, and
// nothing is left to multiply per key.
//
// Values.  O += P V with V = fp16(s (c - z) 2^E_g) and P = fp16(2^7 exp(..)): two
// roundings of 2^-12.  One E_g per CTA serves while V's scales of a group lie
// within four octaves.  (Scales as factors of the weights or scores cost a
// shared-memory word per row and key each: 2.5 times the time, measured.)
//
// The other way.  Where a tile's scales are further apart (K's: over 12 octaves),
// a CTA goes on with operands c - z alone: S_g = Q_g (c - z)_g^T, s_ij = f_i sum_g
// sk_gj S_g,ij in fp32, O_g += W_g (c - z)_g with W_g,ij = fp16(P_ij sv_gj /
// top_gi), and the powers of two `top` per row and group of the attention of a
// few rows over this cache (decode_cache_kernel.cuh, where they are explained).  At the
// first such tile O goes over from E_g to a `top` that its own size allows, since E_g
// says nothing of what the row has weighed.  (With a key 2^-14 of the others in each 700,
// the first two cases below take 36 and 115 us; 35 and 112 with E_g as the first top,
// which lost the weights of small values behind zeros.)
//
// CTA: 640 threads, one per SM.  Warp 0 brings pages into a ring (bulk copies),
// warp 2 looks at a tile's scales, warps 12-19 turn it into K-major and MN-major
// operand tiles (128-byte swizzle), warps 4-7 and 8-11 are two softmax streams
// (thread = row), for which warps 1 and 3 issue the products.  With two row tiles
// (NT = 2) stream t has tile t and both use every key tile; with one (NT = 1) the
// streams take the key tiles in turn, each with accumulators of its own, merged
// at the end, half of the columns by each (the first alone: 31.7 us for the first
// case below, not 30.6).  The softmax takes its scores into registers at once, so
// that the next tile's are made while it works.
//
// Tensor memory, stream t, from column 128 t: the scores in 64, the weights in 32
// and another 32, so that a tile's are put down while the product with the ones
// before still runs.  O in [256 + 128 t, + d_v).  In the other way S_0, S_1 in the
// 128 columns, then the scores over S_0 and W_0, W_1 over S_1, one tile after the
// other.  (Q's rows there, and one place for the weights: the softmax waited 400
// cycles of 2600 a tile for it; a product of 64 columns takes some 54 cycles
// either way.)
//
// A 32-bit word of codes becomes four pairs of operands by one AND-OR and two
// fp16 operations each (0x6400 | c is 1024 + c); the pairs are the dims (k, k + 4)
// of eight, an order that Q's rows are given too and that O's columns lose again
// when they are written.
//
// Measured (GB300, device time of the whole call, and of this kernel beside the
// others').  Widths 128 except the last: 32 sequences of 64-1024 own keys behind
// 8192, 32 heads on 8 (128 rows a head): 30.6 us, 17; the same calls on the warps of
// decode_cache_kernel.cuh 39.7.  64 sequences behind 32768 keys (256 rows): 73 us, 55
// from the end of the own keys' kernel into which it runs; on the warps 190.  16
// sequences, 64 heads on one, behind 16384 (1024 rows): 31.7 us, 19; 51.8.  24
// sequences, 4 queries, 16 heads on 4, behind 5001, widths 128 and 64 (384 rows):
// 32.4 us, 18; 40.4.  The tensor pipe is busy in 11 and 19 % of the cycles of the
// first and the third, the schedulers issue in 39 and 42, and no pipe is above 30:
// a tile takes a stream some 2300 cycles whatever its products take (260), the
// chain of barrier, scores, exponentials (64 of a thread), weights and barrier with
// five warps a scheduler; and a CTA 8000 cycles before its first and 8000 behind
// its last, half of a range of 7 tiles.
// Tried and left out: page numbers 32 at a time and the first pages earlier (0);
// half of O written by the operands' warps (2 % slower); a maximum in place of the
// sum (a seventh slower).
#include <cstdint>
#include <cuda_runtime.h>
#include <type_traits>

#include "cache_mma.cuh"

namespace esd {
namespace {

constexpr float kNoKey = -1e30f;    // the reference (exp2 domain) of a row that has seen no key
constexpr int kLazy = 5, kSlack = 4, kTopBits = 6;      // as in decode_cache_kernel.cuh
static_assert(kLazy + kSlack + kTopBits <= 15, "weights are fp16");
constexpr int kLeastTop = -118, kMostTop = 126;
// Scales that the folded operands take: V's of a group between 2^(X - 2) and
// 2^(X + 2), X the exponent of the CTA's first; K's of a tile 2^12 apart; neither
// beyond 2^+-100.
constexpr int kBelow = 2, kAbove = 1, kSpreadK = 12, kMostExp = 100;
// P 2^kFastBits is fp16: a row's reference moves when a tile's sum of them passes
// 2^15.  (The sum is needed anyway; a maximum of every tile took a seventh of the
// kernel's time.)
constexpr int kFastBits = 7;
constexpr float kMostSum = 32768.0f;
// Where scales come beside the operands O's rows are handed over with their largest
// element below 2^(kHandOver + 1): it is at most 15 times the sum of the weights' products
// of up to 2^31 keys, so that top is at most 2^-5 of the largest of these (2^31 15 2^5 <
// 2^kHandOver), as it is where the weights have been so from the first tile on, or finer.
constexpr int kHandOver = 40;
constexpr int kScaleK = 4;          // K's largest scale becomes 2^4 to 2^5
constexpr int kSumShift = 6;        // sum q_g 2^-6 and s (8 - z) 2^6 are fp16
constexpr int kKeys = 64;           // keys of a tile: two pages
constexpr int kTilePages = kKeys / kPageTokens;

// What the softmax and the products need to know of a tile.
struct __align__(16) TileHead {
  uint32_t mask[2];       // the keys there are, of each page
  float unscale;          // 2^-e of K's operands
  int32_t fast;           // 1: scales in the operands (these four are read as one)
  float up[2];            // fast: the weights' and V's power of two of each group
  float pad[2];
  float most[2][2];       // else: the largest of V's scales, [group][page]
};

template <int DH, int DV, int NT>
struct TileCfg {
  static constexpr int GK = DH / kQuantGroup, GV = DV / kQuantGroup;
  static constexpr int kBlock = page_head_bytes(DH, DV);
  static constexpr int kRawStages = 4, kStages = NT == 2 ? 3 : 4;
  static constexpr int kQTile = 128 * DH * 2, kQx = 128 * 32;
  static constexpr int kK16 = kKeys * DH * 2, kV16 = kKeys * DV * 2, kKx = kKeys * 32;
  static constexpr int kOp = kK16 + kV16 + kKx;
  static constexpr int kScales = (GK + GV) * kKeys * 4;
  static constexpr int kPrep = kScales + kKeys * 4;          // and K's sums' factors
  static constexpr uint32_t kColW = 64;      // of a stream's weights in tensor memory: 32 columns, two of them
  static constexpr int kOffQ = 0;
  static constexpr int kOffOp = kOffQ + NT * kQTile;         // [stage] K16, V16, K's sums
  static constexpr int kOffQx = kOffOp + kStages * kOp;      // [row tile]
  static constexpr int kOffRaw = kOffQx + NT * kQx;
  static constexpr int kOffPrep = kOffRaw + kRawStages * kTilePages * kBlock;    // [raw stage] (scale, z) or scales
  static constexpr int kOffRawHead = kOffPrep + kRawStages * kPrep;            // [raw stage]
  static constexpr int kOffScale = kOffRawHead + kRawStages * static_cast<int>(sizeof(TileHead));   // [stage]
  static constexpr int kOffHead = kOffScale + kStages * kScales;                 // [stage]
  static constexpr int kOffRawMask = kOffHead + kStages * static_cast<int>(sizeof(TileHead));       // [raw stage][2]
  // Of each row, while Q is put down; (l, shift) of both streams (NT = 1).
  static constexpr int kOffState = (kOffRawMask + kRawStages * 8 + 15) / 16 * 16;
  static constexpr int kOffBar = kOffState + NT * 128 * 16;
  static constexpr int kBarRawFull = 0;
  static constexpr int kBarRawEmpty = kBarRawFull + kRawStages;
  static constexpr int kBarPrep = kBarRawEmpty + kRawStages;
  static constexpr int kBarFull = kBarPrep + kRawStages;
  static constexpr int kBarEmpty = kBarFull + kStages;
  static constexpr int kBarS = kBarEmpty + kStages;          // [2]
  static constexpr int kBarSFree = kBarS + 2;                // [2]
  // [2][2], of each place of the weights: a warp may be a tile ahead of the others.
  static constexpr int kBarP = kBarSFree + 2;
  static constexpr int kBarPV = kBarP + 4;
  static constexpr int kBarQ = kBarPV + 4;
  static constexpr int kBarDrain = kBarQ + 1;                // [2]
  static constexpr int kNumBars = kBarDrain + 2;
  static constexpr int kOffTmem = kOffBar + kNumBars * 8;
  static constexpr int kOffAbort = kOffTmem + 4;
  static constexpr int kSmemBytes = kOffAbort + 4 + 1024;    // slack for 1024-byte alignment
  static constexpr int kThreads = 640, kOpThreads = 256;
  // Registers: 96 a thread at launch, moved between the five warpgroups.
  static constexpr uint32_t kRegsLaunch = 96, kRegsControl = 64, kRegsSoftmax = 136, kRegsOperands = 72;
  static_assert(kRegsControl + 2 * kRegsSoftmax + 2 * kRegsOperands <= 5 * kRegsLaunch, "the block's registers");
  static_assert(kSmemBytes <= 232448, "shared memory");
  static_assert(kBlock % 16 == 0 && kOffRaw % 16 == 0 && kOffScale % 16 == 0 && kOffBar % 8 == 0, "alignment");
  static_assert(kOp % 1024 == 0 && kOffOp % 1024 == 0, "swizzled tiles");
  static_assert(NT == 2 || 128 * DV * 4 <= kStages * kOp, "the streams' sums over the operand tiles");
  static_assert(kQTile >= 16384 && kRawStages * kTilePages * kBlock >= 16384, "32 dims of 128 rows on their way out");
};

__device__ __forceinline__ uint32_t hmul2_bits(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hsub2_bits(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The pairs (k, k + 4) of eight codes less a number, as fp16: from 1024 + it (both
// halves) and -(64 + it).
__device__ __forceinline__ uint4 operand8(uint32_t codes, uint32_t z, uint32_t z16) {
  auto low = [&](uint32_t x) { return hsub2_bits((x & 0x000F000Fu) | 0x64006400u, z); };
  auto high = [&](uint32_t x) {                                         // (1024 + 16 c) / 16 - (64 + z)
    return hfma2_bits((x & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, z16);
  };
  return make_uint4(low(codes), high(codes), low(codes >> 8), high(codes >> 8));
}
// ... less the zero point in the lowest byte of `word`.
__device__ __forceinline__ uint4 operand8z(uint32_t codes, uint32_t word) {
  const uint32_t z = __byte_perm(word, 0x64646464u, 0x4040);            // 1024 + z, twice
  return operand8(codes, z, ((z & 0x00FF00FFu) << 4) + 0xD400D400u);
}
__device__ __forceinline__ uint4 times(uint4 x, uint32_t s) {
  return make_uint4(hmul2_bits(x.x, s), hmul2_bits(x.y, s), hmul2_bits(x.z, s), hmul2_bits(x.w, s));
}

// A row's power of two, from the bits of its largest magnitude: 2^14 <= max 2^e <
// 2^15; less below 2^-106, and 0 for 0 and what is not finite.
__device__ __forceinline__ int row_exponent(uint32_t bits) {
  return bits == 0u || bits >= 0x7F800000u ? 0 : min(14 + 127 - static_cast<int>(bits >> 23), 120);
}

// K-major tile without a swizzle: 8 x 8 matrices of 128 bytes, the two of a
// 16-element row next to each other.
__device__ __forceinline__ SmemDesc plain_desc(uint32_t saddr) {
  SmemDesc d = sw128_desc_words(saddr, 128, 256);
  d.hi &= ~(7u << 29);
  return d;
}

// Four products of 16 of the inner dimension, A in tensor memory 8 columns and B
// kStep bytes apart; `accumulate`: the first adds to D.  One election, and the
// operands' places by constants: the issue of a product of its own costs 70
// cycles, more than the tensor core needs for 64 columns.  Called by whole warps.
template <int kStep>
__device__ __forceinline__ void umma_ts_four(uint32_t d, uint32_t a, SmemDesc b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 d0, d1, d2, d3;\n\t.reg .b32 r, b1, b2, b3, a1, a2, a3;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "add.u32 b1, %2, %6;\n\tadd.u32 b2, %2, 2 * %6;\n\tadd.u32 b3, %2, 3 * %6;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
      "mov.b64 d0, {%2, %3};\n\tmov.b64 d1, {b1, %3};\n\tmov.b64 d2, {b2, %3};\n\tmov.b64 d3, {b3, %3};\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], d0, %4, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], d1, %4, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], d2, %4, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], d3, %4, 1;\n\t}\n"
      :: "r"(d), "r"(a), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate), "n"(kStep >> 4) : "memory");
}

// The same with A in shared memory, 32 bytes apart like B.
__device__ __forceinline__ void umma_ss_four(uint32_t d, SmemDesc a, SmemDesc b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 d0, d1, d2, d3, c0, c1, c2, c3;\n\t.reg .b32 r, b1, b2, b3, a1, a2, a3;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "add.u32 b1, %3, 2;\n\tadd.u32 b2, %3, 4;\n\tadd.u32 b3, %3, 6;\n\t"
      "add.u32 a1, %1, 2;\n\tadd.u32 a2, %1, 4;\n\tadd.u32 a3, %1, 6;\n\t"
      "mov.b64 d0, {%3, %4};\n\tmov.b64 d1, {b1, %4};\n\tmov.b64 d2, {b2, %4};\n\tmov.b64 d3, {b3, %4};\n\t"
      "mov.b64 c0, {%1, %2};\n\tmov.b64 c1, {a1, %2};\n\tmov.b64 c2, {a2, %2};\n\tmov.b64 c3, {a3, %2};\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], c0, d0, %5, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], c1, d1, %5, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], c2, d2, %5, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], c3, d3, %5, 1;\n\t}\n"
      :: "r"(d), "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate) : "memory");
}

template <int DH, int DV, int NT>
__global__ void __launch_bounds__(640, 1) prefix_tile_kernel(const __grid_constant__ PrefixTileParams p) {
  using C = TileCfg<DH, DV, NT>;
  constexpr int GK = C::GK, GV = C::GV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int idx) -> uint32_t { return sbase + C::kOffBar + 8 * idx; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffAbort);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffTmem);
  const uint32_t warp = warp_id(), lane = lane_id();

  // ---- work: KV head, rows [r0, r0 + 128 NT), tiles [t0, t0 + n) of the prefix ----
  const int item = static_cast<int>(blockIdx.x);
  const int split = item % p.splits, block = item / p.splits;
  const int h = block / p.row_blocks, r0 = (block - h * p.row_blocks) * 128 * NT;
  const int R = p.B * p.per;
  const int cap = p.prefix_pages * kPageTokens;
  int len = *p.length;
  if (item == 0 && threadIdx.x == 0 && len > cap) record_status(p.status, ATTN_ERR_PAGE);
  len = len < 0 ? 0 : (len > cap ? cap : len);
  const int tiles = len / kKeys + (len % kKeys != 0);
  const int each = (tiles + p.splits - 1) / p.splits;
  if (item == 0 && threadIdx.x == 0) *p.used = each > 0 ? (tiles + each - 1) / each : 0;
  const int t0 = split * each;
  const int n = tiles - t0 < each ? tiles - t0 : each;
  if (n <= 0) {                // (the whole CTA, before it owns anything)
    cudaGridDependencySynchronize();
    return;
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kRawStages; ++s) {
      mbar_init(bar(C::kBarRawFull + s), 1);
      mbar_init(bar(C::kBarRawEmpty + s), C::kOpThreads);
      mbar_init(bar(C::kBarPrep + s), 1);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar(C::kBarFull + s), C::kOpThreads);
      mbar_init(bar(C::kBarEmpty + s), NT);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(C::kBarS + t), 1);
      mbar_init(bar(C::kBarSFree + t), 128);
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(C::kBarP + 2 * t + i), 128);
        mbar_init(bar(C::kBarPV + 2 * t + i), 1);
      }
      mbar_init(bar(C::kBarDrain + t), 1);
    }
    mbar_init(bar(C::kBarQ), 256);
    fence_mbar_init();
    *abort_flag = status_blocks(p.status) ? 2 : 0;
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const uint64_t limit = p.wait_limit_ns;
  auto wait = [&](int idx, uint32_t parity) { return mbar_wait(bar(idx), parity, abort_flag, limit); };
  auto wait_all = [&](int idx, uint32_t parity) { return __all_sync(0xffffffffu, wait(idx, parity)); };
  // Key tiles of stream t: the k-th is tile tile_of(t, k).
  auto tile_of = [](int t, int k) { return NT == 2 ? k : 2 * k + t; };
  auto count_of = [&](int t) { return NT == 2 ? n : (n + 1 - t) / 2; };
  auto phase = [](int t, int stages) { return static_cast<uint32_t>((t / stages) & 1); };

  // ---- Q: each row's power of two, its fp16 operands and sums, by warps 4-19 ----
  // 16 bytes a lane, 256 / D rows of a warp at a time, put down swizzled.
  if (warp >= 4) {
    constexpr int kLanes = DH / 8, kAt = 32 / kLanes, kWarpRows = 128 * NT / 16, kTimes = kWarpRows / kAt;
    const int c = static_cast<int>(lane) % kLanes;
    const int first = (static_cast<int>(warp) - 4) * kWarpRows + static_cast<int>(lane) / kLanes;
    uint4 v[kTimes];
    int of = (r0 + first) / p.per, rem = r0 + first - of * p.per;
#pragma unroll
    for (int i = 0; i < kTimes; ++i) {
      const int64_t at = (static_cast<int64_t>(of) * p.Hkv + h) * p.per + rem;
      v[i] = r0 + first + i * kAt < R ? reinterpret_cast<const uint4*>(p.Q)[at * kLanes + c] : make_uint4(0u, 0u, 0u, 0u);
      rem += kAt;
#pragma unroll
      for (int o = 0; o < kAt; ++o)
        if (rem >= p.per) rem -= p.per, ++of;
    }
    // (Each step for all rows, so that their shuffles overlap.)
    uint32_t mb[kTimes];
    float sum[kTimes];
#pragma unroll
    for (int i = 0; i < kTimes; ++i) mb[i] = __float_as_uint(bf16_absmax_value(bf16_absmax_fold(0u, v[i])));
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1)
#pragma unroll
      for (int i = 0; i < kTimes; ++i) mb[i] = max(mb[i], __shfl_xor_sync(0xffffffffu, mb[i], off));
#pragma unroll
    for (int i = 0; i < kTimes; ++i) {
      const int rr = first + i * kAt, in_tile = rr & 127;
      const float times_e = exp2_int(row_exponent(mb[i]));
      const uint4 u = bf16x8_to_f16x8_scaled(v[i], times_e);
      *reinterpret_cast<uint4*>(smem + C::kOffQ + rr / 128 * C::kQTile + c / 8 * (128 * 128) + in_tile * 128 +
                                (((c & 7) ^ (rr & 7)) * 16)) =
          make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632), __byte_perm(u.y, u.w, 0x5410),
                     __byte_perm(u.y, u.w, 0x7632));
      const uint32_t xs[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int o = 0; o < 4; ++o) a = fmaf(bf16_lo(xs[o]), times_e, a), b = fmaf(bf16_hi(xs[o]), times_e, b);
      sum[i] = a + b;
    }
#pragma unroll
    for (int off = 4; off > 0; off >>= 1)
#pragma unroll
      for (int i = 0; i < kTimes; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], off);
    // Of each row: sum q_g and the largest magnitude.
    float(*rows_of)[4] = reinterpret_cast<float(*)[4]>(smem + C::kOffState);
#pragma unroll
    for (int i = 0; i < kTimes; ++i) {
      if ((c & 7) == 0) rows_of[first + i * kAt][c / 8] = sum[i];
      if (c == 0) rows_of[first + i * kAt][2] = __uint_as_float(mb[i]);
    }
    fence_proxy_async_smem();
  }

  if (warp < 4) {
    setmaxnreg_to<C::kRegsControl, C::kRegsLaunch>();
    if (warp == 0) {
      // ================= pages into the ring =================
      if (lane == 0 && *abort_flag == 0) {
        int issued = 0;
        for (int j = 0; j < n; ++j) {
          const int st = j % C::kRawStages;
          if (j >= C::kRawStages && !wait(C::kBarRawEmpty + st, phase(j - C::kRawStages, C::kRawStages))) break;
          uint32_t* mask = reinterpret_cast<uint32_t*>(smem + C::kOffRawMask) + 2 * st;
          const uint8_t* src[kTilePages];
          int bytes = 0;
#pragma unroll
          for (int i = 0; i < kTilePages; ++i) {
            const int page = (t0 + j) * kTilePages + i;
            const int64_t left = len - static_cast<int64_t>(page) * kPageTokens;
            src[i] = nullptr;
            mask[i] = left >= kPageTokens ? 0xFFFFFFFFu : left > 0 ? (1u << left) - 1u : 0u;
            if (left <= 0) continue;
            const int id = p.table[page];
            if (id < 0 || id >= p.pages) {
              record_status(p.status, ATTN_ERR_PAGE);
              mask[i] = 0u;
              continue;
            }
            src[i] = p.pool + (static_cast<int64_t>(id) * p.Hkv + h) * C::kBlock;
            bytes += C::kBlock;
          }
          mbar_arrive_expect_tx(bar(C::kBarRawFull + st), bytes);
#pragma unroll
          for (int i = 0; i < kTilePages; ++i)
            if (src[i])
              bulk_load(sbase + C::kOffRaw + (st * kTilePages + i) * C::kBlock, src[i], C::kBlock,
                        bar(C::kBarRawFull + st));
          ++issued;
        }
        if (*abort_flag) {
          // Every copy already in flight must land before the CTA can exit.
          int no_abort = 0;
          for (int j = issued > C::kRawStages ? issued - C::kRawStages : 0; j < issued; ++j)
            mbar_wait(bar(C::kBarRawFull + j % C::kRawStages), phase(j, C::kRawStages), &no_abort, limit);
        }
      }
    } else if (warp == 1 || warp == 3) {
      // ================= products =================
      const int t = warp == 1 ? 0 : 1, count = count_of(t);
      if (__all_sync(0xffffffffu, *abort_flag == 0) && count > 0) {
        constexpr uint32_t kIdQK = idesc_f16_f32(128, kKeys, false, false);
        constexpr uint32_t kIdPV = idesc_f16_f32(128, DV, false, true), kIdPVg = idesc_f16_f32(128, 64, false, true);
        constexpr int kStep = NT == 2 ? 1 : 2;
        const SmemDesc dq = sw128_desc_words(sbase + C::kOffQ + (NT == 2 ? t : 0) * C::kQTile, 16, 1024);
        const SmemDesc dqx = plain_desc(sbase + C::kOffQx + (NT == 2 ? t : 0) * C::kQx);
        const SmemDesc dk0 = sw128_desc_words(sbase + C::kOffOp, 16, 1024);
        const SmemDesc dv0 = sw128_desc_words(sbase + C::kOffOp + C::kK16, kKeys * 128, 1024);
        const SmemDesc dx0 = plain_desc(sbase + C::kOffOp + C::kK16 + C::kV16);
        const uint32_t tS = tmem + 128 * t, tO = tmem + 256 + 128 * t;
        auto fast_tile = [&](int st) {
          return __shfl_sync(0xffffffffu, reinterpret_cast<const TileHead*>(smem + C::kOffHead)[st].fast, 0) != 0;
        };
        auto scores = [&](int st, bool fast) {     // of the tile in stage st
          const SmemDesc dk = desc_step(dk0, st * C::kOp);
          if (fast) {
#pragma unroll
            for (int g = 0; g < GK; ++g) {
              const SmemDesc dkg = desc_step(dk, g * kKeys * 128);
              umma_ss_four(tS, desc_step(dq, g * 128 * 128), dkg, kIdQK, g > 0 ? 1u : 0u);
            }
            umma_ss_we(tS, dqx, desc_step(dx0, st * C::kOp), kIdQK, 1u);
          } else {
#pragma unroll 1
            for (int g = 0; g < GK; ++g)
              umma_ss_four(tS + 64 * g, desc_step(dq, g * 128 * 128), desc_step(dk, g * kKeys * 128), kIdQK, 0u);
          }
          umma_commit_we(bar(C::kBarS + t));
        };
        // Stage and phase of the tile at hand and of the next.
        int st = NT == 2 ? 0 : t;
        uint32_t ph = 0;
        bool ok = wait_all(C::kBarQ, 0) && wait_all(C::kBarFull + st, ph), fast = true;
        if (ok) {
          tc_fence_after_sync();
          fast = fast_tile(st);
          scores(st, fast);
        }
        for (int k = 0; k < count && ok; ++k) {
          int next = st + kStep;
          uint32_t next_ph = ph;
          if (next >= C::kStages) next -= C::kStages, next_ph ^= 1u;
          bool next_fast = false;
          if (k + 1 < count) {
            ok = wait_all(C::kBarFull + next, next_ph);
            if (!ok) break;
            next_fast = fast_tile(next);
            if (next_fast) {                     // as soon as the scores before have been read
              ok = wait_all(C::kBarSFree + t, static_cast<uint32_t>(k & 1));
              if (!ok) break;
              tc_fence_after_sync();
              scores(next, true);
            }
          }
          ok = wait_all(C::kBarP + 2 * t + (k & 1), static_cast<uint32_t>((k >> 1) & 1));
          if (!ok) break;
          tc_fence_after_sync();
          const SmemDesc dv = desc_step(dv0, st * C::kOp);
          if (fast) {
            umma_ts_four<2048>(tO, tS + C::kColW + 32 * (k & 1), dv, kIdPV, k > 0 ? 1u : 0u);
          } else {
#pragma unroll 1
            for (int g = 0; g < GV; ++g)
              umma_ts_four<2048>(tO + 64 * g, tS + 64 + 32 * g, desc_step(dv, g * kKeys * 128), kIdPVg, k > 0 ? 1u : 0u);
          }
          umma_commit_we(bar(C::kBarPV + 2 * t + (k & 1)));
          umma_commit_we(bar(C::kBarEmpty + st));
          if (k + 1 < count && !next_fast) scores(next, false);     // (over the weights just used)
          st = next, ph = next_ph, fast = next_fast;
        }
        int no_abort = 0;
        umma_commit_we(bar(C::kBarDrain + t));
        mbar_wait(bar(C::kBarDrain + t), 0, &no_abort, limit);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ================= scales =================
      bool ok = *abort_flag == 0, fast = true;
      int x[GV];                             // exponents of V's scales, 0 before the first
      bool set[GV];
#pragma unroll
      for (int g = 0; g < GV; ++g) x[g] = 0, set[g] = false;
      for (int j = 0; j < n && ok; ++j) {
        const int rs = j % C::kRawStages;
        ok = wait_all(C::kBarRawFull + rs, phase(j, C::kRawStages));
        if (!ok) break;
        const uint8_t* raw = smem + C::kOffRaw + rs * kTilePages * C::kBlock;
        const uint32_t* masks = reinterpret_cast<const uint32_t*>(smem + C::kOffRawMask) + 2 * rs;
        TileHead& head = reinterpret_cast<TileHead*>(smem + C::kOffRawHead)[rs];
        uint32_t word[GK + GV][kTilePages];    // of key `lane` of each page; 0 for keys that are not there
        uint32_t most[GK + GV][kTilePages], all[GK + GV], least[GK + GV];
#pragma unroll
        for (int w = 0; w < GK + GV; ++w) {
          least[w] = 0xFFFFFFFFu;
#pragma unroll
          for (int i = 0; i < kTilePages; ++i) {
            const uint8_t* words = raw + i * C::kBlock + (w < GK ? off_k_words(DH, DV) : off_v_words(DH, DV));
            const int of = w < GK ? static_cast<int>(lane) * GK + w : static_cast<int>(lane) * GV + w - GK;
            word[w][i] = (masks[i] >> lane) & 1u ? reinterpret_cast<const uint32_t*>(words)[of] : 0u;
            const uint32_t scale = word[w][i] & 0xFFFF0000u;
            most[w][i] = __reduce_max_sync(0xffffffffu, scale);
            least[w] = min(least[w], scale ? scale : 0xFFFFFFFFu);
          }
          least[w] = __reduce_min_sync(0xffffffffu, least[w]);
          all[w] = max(most[w][0], most[w][1]);
        }
        uint32_t k_most = all[0], k_least = least[0];
        if (GK == 2) k_most = max(k_most, all[GK - 1]), k_least = min(k_least, least[GK - 1]);
        // Exponents of the bits of a scale (those of 0 do not count).
        auto exponent = [](uint32_t bits) { return static_cast<int>(bits >> 23) - 127; };
        const int k_exp = k_most ? exponent(k_most) : 0;
        fast = fast && (!k_most || (k_exp <= kMostExp && k_exp >= -kMostExp && exponent(k_least) >= k_exp - kSpreadK));
#pragma unroll
        for (int g = 0; g < GV; ++g) {
          if (all[GK + g] == 0u) continue;
          const int hi = exponent(all[GK + g]), lo = exponent(least[GK + g]);
          if (!set[g]) x[g] = hi, set[g] = true;
          fast = fast && hi <= kMostExp && hi >= -kMostExp && hi <= x[g] + kAbove && lo >= x[g] - kBelow;
        }
        uint32_t* prep = reinterpret_cast<uint32_t*>(smem + C::kOffPrep + rs * C::kPrep) + lane;
#pragma unroll
        for (int w = 0; w < GK + GV; ++w)
#pragma unroll
          for (int i = 0; i < kTilePages; ++i) {
            const float scale = bf16_hi(word[w][i]);
            // (bf16 has 16 bits, so that the zero point has a place beside it too.)
            uint32_t out = word[w][i];
            if (fast) out = pack_half2(0.f, scale * exp2_int(w < GK ? kScaleK - k_exp : -x[w < GK ? 0 : w - GK])) |
                            (word[w][i] & 0xFFu);
            prep[w * kKeys + i * kPageTokens] = out;
          }
        if (fast) {                              // s (8 - z) 2^kSumShift of both groups
#pragma unroll
          for (int i = 0; i < kTilePages; ++i) {
            float x[2] = {0.f, 0.f};
#pragma unroll
            for (int g = 0; g < GK; ++g)
              x[g] = bf16_hi(word[g][i]) * exp2_int(kScaleK + kSumShift - k_exp) *
                     static_cast<float>(8 - static_cast<int>(word[g][i] & 0xFFu));
            prep[(GK + GV) * kKeys + i * kPageTokens] = pack_half2(x[0], x[1]);
          }
        }
        if (lane == 0) {
          head.mask[0] = masks[0], head.mask[1] = masks[1];
          head.unscale = exp2_int(k_exp - kScaleK);
          head.fast = fast ? 1 : 0;
#pragma unroll
          for (int g = 0; g < GV; ++g) {
            head.up[g] = exp2_int(kFastBits - x[g]);
#pragma unroll
            for (int i = 0; i < kTilePages; ++i) head.most[g][i] = __uint_as_float(most[GK + g][i]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kBarPrep + rs));
      }
    }
  } else if (warp >= 12) {
    // ================= codes into operands =================
    asm volatile("bar.arrive 2, 512;" ::: "memory");
    setmaxnreg_to<C::kRegsOperands, C::kRegsLaunch>();
    const int tid = static_cast<int>(threadIdx.x) - 384, w8 = static_cast<int>(warp) - 12;
    // The second half of the sums' inner step is 0.
    for (int i = tid; i < C::kStages * kKeys; i += C::kOpThreads)
      *reinterpret_cast<uint4*>(smem + C::kOffOp + i / kKeys * C::kOp + C::kK16 + C::kV16 + i % kKeys / 8 * 256 + 128 +
                                i % 8 * 16) = make_uint4(0u, 0u, 0u, 0u);
    bool ok = *abort_flag == 0;
    int st = C::kStages - 1;
    uint32_t ph = 0;                       // of the stage's next release
    for (int j = 0; j < n && ok; ++j) {
      const int rs = j % C::kRawStages;
      if (++st == C::kStages) st = 0, ph ^= 1u;
      ok = wait_all(C::kBarRawFull + rs, phase(j, C::kRawStages)) && wait_all(C::kBarPrep + rs, phase(j, C::kRawStages));
      if (ok && j >= C::kStages) ok = wait_all(C::kBarEmpty + st, ph);
      if (!ok) break;
      const uint8_t* raw = smem + C::kOffRaw + rs * kTilePages * C::kBlock;
      const uint32_t* prep = reinterpret_cast<const uint32_t*>(smem + C::kOffPrep + rs * C::kPrep);
      const TileHead& head = reinterpret_cast<const TileHead*>(smem + C::kOffRawHead)[rs];
      uint8_t* op = smem + C::kOffOp + st * C::kOp;
      const bool fast = head.fast != 0;
      // A row of D dims is D / 8 words; a warp takes 256 / D rows at a time, all of
      // its words requested before the first is converted.
      auto convert = [&](auto width, int codes_at, const uint32_t* scale, uint8_t* out, auto&& operand) {
        constexpr int D = decltype(width)::value, kWords = D / 8, kRows = 32 / kWords, kTimes = kKeys / (8 * kRows);
        const int c = static_cast<int>(lane) % kWords, g = c / 8;
        const int key0 = w8 * kRows + static_cast<int>(lane) / kWords;
        uint8_t* to = out + g * (kKeys * 128);
        uint32_t codes[kTimes], word[kTimes];
#pragma unroll
        for (int i = 0; i < kTimes; ++i) {
          const int key = i * 8 * kRows + key0;
          codes[i] = *reinterpret_cast<const uint32_t*>(raw + key / kPageTokens * C::kBlock + codes_at +
                                                        key % kPageTokens * (D / 2) + 4 * c);
          word[i] = scale[g * kKeys + key];
        }
#pragma unroll
        for (int i = 0; i < kTimes; ++i) {
          const int key = i * 8 * kRows + key0;
          *reinterpret_cast<uint4*>(to + key * 128 + (((c & 7) ^ (key & 7)) * 16)) = operand(codes[i], word[i]);
        }
      };
      constexpr std::integral_constant<int, DH> kDH{};
      constexpr std::integral_constant<int, DV> kDV{};
      if (fast) {
        convert(kDH, off_k_codes(), prep, op, [](uint32_t codes, uint32_t word) {
          return times(operand8(codes, 0x64086408u, 0xD480D480u), __byte_perm(word, 0u, 0x3232));
        });
        convert(kDV, off_v_codes(DH), prep + GK * kKeys, op + C::kK16, [](uint32_t codes, uint32_t word) {
          return times(operand8z(codes, word), __byte_perm(word, 0u, 0x3232));
        });
      } else {
        convert(kDH, off_k_codes(), prep, op, operand8z);
        convert(kDV, off_v_codes(DH), prep + GK * kKeys, op + C::kK16, operand8z);
      }
      if (fast) {
        if (tid < kKeys) {                      // s (8 - z) of each group, three times
          const uint32_t x = prep[(GK + GV) * kKeys + tid];
          *reinterpret_cast<uint4*>(op + C::kK16 + C::kV16 + tid / 8 * 256 + tid % 8 * 16) =
              make_uint4(__byte_perm(x, 0u, 0x1010), x, __byte_perm(x, 0u, 0x3232), 0u);
        }
      } else {
        uint32_t* scales = reinterpret_cast<uint32_t*>(smem + C::kOffScale + st * C::kScales);
        for (int i = tid; i < (GK + GV) * kKeys; i += C::kOpThreads) scales[i] = prep[i] & 0xFFFF0000u;
      }
      if (tid < static_cast<int>(sizeof(TileHead) / 4))
        reinterpret_cast<uint32_t*>(smem + C::kOffHead + st * sizeof(TileHead))[tid] =
            reinterpret_cast<const uint32_t*>(&head)[tid];
      fence_proxy_async_smem();
      mbar_arrive(bar(C::kBarFull + st));
      mbar_arrive(bar(C::kBarRawEmpty + rs));
    }
  } else {
    // ================= softmax =================
    setmaxnreg_to<C::kRegsSoftmax, C::kRegsLaunch>();
    const int t = static_cast<int>(warp) / 4 - 1;          // stream
    const uint32_t quad = warp & 3;
    const int row = static_cast<int>(quad * 32 + lane), tile0 = r0 + (NT == 2 ? 128 * t : 0), r = tile0 + row;
    const bool valid = r < R;
    const uint32_t lane_base = (quad * 32u) << 16;
    const uint32_t tS = tmem + lane_base + 128 * t, tO = tmem + lane_base + 256 + 128 * t;
    // ---- this thread's row of Q: its factor and its sums' operand ----
    float f;
    {
      named_bar_sync(2, 512);                              // (all rows are there)
      {
        const float4 of = reinterpret_cast<const float4*>(smem + C::kOffState)[(NT == 2 ? 128 * t : 0) + row];
        const uint32_t mb = __float_as_uint(of.z);
        // (Not 0, which a masked -inf must not meet; NaN for a row that is not finite.)
        f = fmaxf(p.scale_log2 * exp2_int(-row_exponent(mb)), 0x1p-126f);
        if (mb >= 0x7F800000u) f = __uint_as_float(0x7FC00000u);
        if (NT == 2 || t == 0) {                           // sum q_g 2^-6: three fp16 numbers of each group
          uint32_t h16[6] = {0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
          for (int g = 0; g < GK; ++g) {
            float left = (g == 0 ? of.x : of.y) * exp2_int(-kSumShift);
#pragma unroll
            for (int o = 0; o < 3; ++o) {
              const __half x = __float2half_rn(left);
              left -= __half2float(x);
              h16[3 * g + o] = __half_as_ushort(x);
            }
          }
          uint4* to = reinterpret_cast<uint4*>(smem + C::kOffQx + (NT == 2 ? t : 0) * C::kQx + row / 8 * 256 + row % 8 * 16);
          to[0] = make_uint4(h16[0] | h16[1] << 16, h16[2] | h16[3] << 16, h16[4] | h16[5] << 16, 0u);
          to[8] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      tc_fence_before_sync();
      mbar_arrive(bar(C::kBarQ));
    }
    // Less the reference that P is relative to; the sum of P, times 2^kFastBits
    // until the first tile without folded scales.
    float shift = -kNoKey, l_sum = 0.f;
    // 1 / top, of the folded operands or each row's; the scale from which on a
    // weight may be too large.
    float up[GV], s_lim[GV];
#pragma unroll
    for (int g = 0; g < GV; ++g) up[g] = exp2_int(-kLeastTop), s_lim[g] = 0.f;
    bool folded = true;
    const int mine = count_of(t);
    bool ok = *abort_flag == 0;
    // O's columns of each group times a factor, once the products before have been added.
    auto rescale = [&](int k, float back0, float back1) {
      if (!wait_all(C::kBarPV + 2 * t + ((k - 1) & 1), static_cast<uint32_t>(((k - 1) >> 1) & 1))) return false;
      tc_fence_after_sync();
#pragma unroll 1
      for (int c = 0; c < DV; c += 16) {
        const float times_b = c < 64 ? back0 : back1;
        uint32_t o[16];
        tmem_ld16_nowait(tO + c, o);
        tmem_wait_ld16(o);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * times_b);
        tmem_st16_nowait(tO + c, o);
      }
      return true;
    };
    // The first tile with its scales beside the operands: the power of two that O carries
    // becomes each row's top, as low as O's largest element allows.  (It says nothing of
    // what a row has weighed: its values may have been 0, or its reference have risen since.)
    auto hand_over = [&](int k) {
      if (!wait_all(C::kBarPV + 2 * t + ((k - 1) & 1), static_cast<uint32_t>(((k - 1) >> 1) & 1))) return false;
      tc_fence_after_sync();
      float most[GV], times[GV], again[GV];
#pragma unroll
      for (int g = 0; g < GV; ++g) most[g] = 0.f;
#pragma unroll 1
      for (int c = 0; c < DV; c += 16) {
        uint32_t o[16];
        tmem_ld16_nowait(tO + c, o);
        tmem_wait_ld16(o);
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(__uint_as_float(o[i])));
        if (c < 64) most[0] = fmaxf(most[0], m);
        else most[GV - 1] = fmaxf(most[GV - 1], m);
      }
#pragma unroll
      for (int g = 0; g < GV; ++g) {
        const int was = static_cast<int>(__float_as_uint(up[g]) >> 23) - 127;
        const int room = kHandOver + 127 - static_cast<int>(__float_as_uint(most[g]) >> 23);
        const int by = max(0, min(most[g] > 0.f ? room : -kLeastTop - was, -kLeastTop - was));
        times[g] = exp2_int(min(by, 100)), again[g] = exp2_int(by - min(by, 100));      // (up to 211 octaves)
        up[g] = exp2_int(was + by);
      }
#pragma unroll 1
      for (int c = 0; c < DV; c += 16) {
        const float times_b = c < 64 ? times[0] : times[GV - 1], again_b = c < 64 ? again[0] : again[GV - 1];
        uint32_t o[16];
        tmem_ld16_nowait(tO + c, o);
        tmem_wait_ld16(o);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * times_b * again_b);
        tmem_st16_nowait(tO + c, o);
      }
      tmem_wait_st();                          // (rescale may read it next)
      return true;
    };
    auto row_max = [](const float* s) {
      float m[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int i = 4; i < kKeys - 4; i += 8)
#pragma unroll
        for (int o = 0; o < 4; ++o) m[o] = fmax3(m[o], s[i + 2 * o], s[i + 2 * o + 1]);
      return fmax3(fmax3(m[0], m[1], s[kKeys - 1]), fmax3(m[2], m[3], s[kKeys - 2]), fmaxf(s[kKeys - 3], s[kKeys - 4]));
    };
    // -inf for the keys that are not there.
    auto hide = [&](uint2 mask) {
#pragma unroll 1
      for (int c = 0; c < kKeys; c += 16) {
        uint32_t a[16];
        tmem_ld16_nowait(tS + c, a);
        tmem_wait_ld16(a);
        const uint32_t bits = (c < 32 ? mask.x : mask.y) >> (c & 31);
#pragma unroll
        for (int i = 0; i < 16; ++i) a[i] = (bits >> i) & 1u ? a[i] : 0xFF800000u;
        tmem_st16_nowait(tS + c, a);
      }
      tmem_wait_st();
    };
    int st = NT == 2 ? -1 : t - 2;             // stage of the tile at hand, and its phase
    uint32_t ph = 0;
    for (int k = 0; k < mine && ok; ++k) {
      st += NT == 2 ? 1 : 2;
      if (st >= C::kStages) st -= C::kStages, ph ^= 1u;
      ok = wait_all(C::kBarFull + st, ph);
      if (!ok) break;
      // What is known of the tile is read before its scores are there: the tensor
      // core's operands fill shared memory's pipe, and a word takes hundreds of cycles.
      const TileHead& head = reinterpret_cast<const TileHead*>(smem + C::kOffHead)[st];
      const uint4 known = *reinterpret_cast<const uint4*>(&head);
      const float2 tile_up = *reinterpret_cast<const float2*>(head.up);
      const uint2 mask = make_uint2(known.x, known.y);
      const float unscale = __uint_as_float(known.z);
      const bool fast = __shfl_sync(0xffffffffu, known.w, 0) != 0u;
      ok = wait_all(C::kBarS + t, static_cast<uint32_t>(k & 1));
      if (!ok) break;
      tc_fence_after_sync();
      if (fast) {
        // ---- scales in the operands ----
        if ((mask.x & mask.y) != 0xFFFFFFFFu) hide(mask);
        float s[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) tmem_ld32_nowait(tS + c, reinterpret_cast<uint32_t(&)[32]>(s[c]));
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) tmem_wait_ld32(reinterpret_cast<uint32_t(&)[32]>(s[c]));
        tc_fence_before_sync();
        mbar_arrive(bar(C::kBarSFree + t));
        float fk = f * unscale;              // (not 0, as f)
        fk = fk < 0x1p-126f ? 0x1p-126f : fk;
        // The reference to the row's maximum, where that is above it.
        auto move_reference = [&] {
          const float m = ceilf(row_max(s) * fk);
          float alpha = 1.f;
          if (m + shift > 0.f) {                           // (whole octaves: alpha is a power of two)
            alpha = fast_exp2(-shift - m);
            shift = -m;
          }
          l_sum *= alpha;
          return k == 0 || !__any_sync(0xffffffffu, alpha != 1.f) || rescale(k, alpha, alpha);
        };
        if (k == 0) move_reference();
        if (k > 1) {                             // the weights two tiles before have been used
          ok = wait_all(C::kBarPV + 2 * t + (k & 1), static_cast<uint32_t>(((k >> 1) - 1) & 1));
          if (!ok) break;
          tc_fence_after_sync();
        }
        float l[2];
#pragma unroll 1
        for (int again = 0; again < 2; ++again) {
          const float add = shift + static_cast<float>(kFastBits);
          l[0] = l[1] = 0.f;
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float e0, e1;
              ffma2(e0, e1, s[c + i], s[c + i + 1], fk, fk, add, add);
              e0 = fast_exp2(e0);
              e1 = fast_exp2(e1);
              fadd2(l[0], l[1], e0, e1);
              w[i / 2] = pack_half2(e0, e1);
            }
            tmem_st16_nowait(tS + C::kColW + 32 * (k & 1) + c / 2, w);
          }
          // (Once more at most: with the reference at its maximum a row's sum is at most 2^13.)
          if (!__any_sync(0xffffffffu, l[0] + l[1] > kMostSum)) break;
          tmem_wait_st();                        // (two stores to one place have no order of their own)
          ok = move_reference();
          if (!ok) break;
        }
        if (!ok) break;
        l_sum += l[0] + l[1];
        up[0] = tile_up.x;
        if (GV == 2) up[GV - 1] = tile_up.y;
      } else {
        // ---- scales beside the operands ----
        const float* scales = reinterpret_cast<const float*>(smem + C::kOffScale + st * C::kScales);
        const float* sv = scales + GK * kKeys;
        if (folded) {
          folded = false;
          l_sum *= exp2_int(-kFastBits);
          ok = k == 0 || hand_over(k);
          if (!ok) break;
        }
        // The scores put together, over S_0, and their maximum; then W in the next
        // 64 columns.  (Loops: this is not where the time goes.)
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < kKeys; c += 16) {
          uint32_t a[16], b[16];
          tmem_ld16_nowait(tS + c, a);
          if (GK == 2) tmem_ld16_nowait(tS + 64 + c, b);
          tmem_wait_ld16(a);
          if (GK == 2) tmem_wait_ld16(b);
          const uint32_t bits = (c < 32 ? mask.x : mask.y) >> (c & 31);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x = __uint_as_float(a[i]) * scales[c + i];
            if (GK == 2) x = fmaf(__uint_as_float(b[i]), scales[kKeys + c + i], x);
            if (!((bits >> i) & 1u)) x = -INFINITY;
            mx = fmaxf(mx, x);
            a[i] = __float_as_uint(x);
          }
          tmem_st16_nowait(tS + c, a);
        }
        tmem_wait_st();
        bool need = fmaf(mx, f, shift) > static_cast<float>(kLazy);
#pragma unroll
        for (int g = 0; g < GV; ++g) need |= fmaxf(head.most[g][0], head.most[g][1]) > s_lim[g];
        if (__any_sync(0xffffffffu, need)) {
          const float m = ceilf(mx * f);
          float alpha = 1.f;
          if (m + shift > static_cast<float>(kLazy)) {
            alpha = fast_exp2(-shift - m);
            shift = -m;
          }
          l_sum *= alpha;
          float most[GV], back[GV];
          bool change = false;
#pragma unroll
          for (int g = 0; g < GV; ++g) most[g] = 0.f;
#pragma unroll 1
          for (int c = 0; c < kKeys; c += 16) {
            uint32_t a[16];
            tmem_ld16_nowait(tS + c, a);
            tmem_wait_ld16(a);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float w = fast_exp2(fmaf(__uint_as_float(a[i]), f, shift));
#pragma unroll
              for (int g = 0; g < GV; ++g) most[g] = fmaxf(most[g], w * sv[g * kKeys + c + i]);
            }
          }
#pragma unroll
          for (int g = 0; g < GV; ++g) {
            const float was = alpha * inverse_power(up[g]);
            const uint32_t at_least = max(near_power(was), static_cast<uint32_t>(127 + kLeastTop) << 23);
            const uint32_t now = max(at_least, next_power(most[g] * exp2_int(-kTopBits)));
            const float top = __uint_as_float(min(now, static_cast<uint32_t>(127 + kMostTop) << 23));
            up[g] = inverse_power(top);
            back[g] = was * up[g];                           // at most 1
            s_lim[g] = top * exp2_int(kTopBits + kSlack);
            change |= back[g] != 1.f;
          }
          if (k > 0 && __any_sync(0xffffffffu, change)) {
            ok = rescale(k, back[0], back[GV - 1]);
            if (!ok) break;
          }
        }
#pragma unroll 1
        for (int c = 0; c < kKeys; c += 16) {
          uint32_t a[16], w[GV][8];
          tmem_ld16_nowait(tS + c, a);
          tmem_wait_ld16(a);
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float e0 = fast_exp2(fmaf(__uint_as_float(a[i]), f, shift));
            const float e1 = fast_exp2(fmaf(__uint_as_float(a[i + 1]), f, shift));
            l_sum += e0 + e1;
#pragma unroll
            for (int g = 0; g < GV; ++g)
              w[g][i / 2] = pack_half2(e0 * up[g] * sv[g * kKeys + c + i], e1 * up[g] * sv[g * kKeys + c + i + 1]);
          }
#pragma unroll
          for (int g = 0; g < GV; ++g) tmem_st8_nowait(tS + 64 + 32 * g + c / 2, w[g]);
        }
      }
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive(bar(C::kBarP + 2 * t + (k & 1)));
    }
    if (folded) l_sum *= exp2_int(-kFastBits);
    cudaTriggerProgrammaticLaunchCompletion();     // the merge kernel may start (it waits for this grid)
    if (ok && mine > 0) ok = wait_all(C::kBarPV + 2 * t + ((mine - 1) & 1), static_cast<uint32_t>(((mine - 1) >> 1) & 1));
    tc_fence_after_sync();
    float weight = 1.f, other = 0.f;           // of this stream's sums and of the other's (NT = 1)
    float* theirs = reinterpret_cast<float*>(smem + C::kOffOp);        // [dim][row], over the operand tiles
    // The columns of O that this stream writes: NT = 1, half of them.
    const int c0 = NT == 2 ? 0 : t * (DV / 2), c1 = NT == 2 ? DV : c0 + DV / 2;
    if constexpr (NT == 1) {
      // Both streams' products are done: each hands the other its sums of the other's half.
      named_bar_sync(1, 256);
      float2* state = reinterpret_cast<float2*>(smem + C::kOffState);
      state[t * 128 + row] = make_float2(l_sum, shift);
      const float down = inverse_power(up[t == 0 ? GV - 1 : 0]);
#pragma unroll 1
      for (int c = DV / 2 - c0; c < DV - c0; c += 16) {
        uint32_t o[16];
        tmem_ld16_nowait(tO + c, o);
        tmem_wait_ld16(o);
#pragma unroll
        for (int i = 0; i < 16; ++i) theirs[(c + i) * 128 + row] = mine > 0 ? __uint_as_float(o[i]) * down : 0.f;
      }
      named_bar_sync(1, 256);
      const float2 x = state[(1 - t) * 128 + row];
      const float ref = fminf(shift, x.y);     // less the larger reference
      weight = fast_exp2(ref - shift);
      other = fast_exp2(ref - x.y);
      l_sum = t == 0 ? l_sum * weight + x.x * other : x.x * other + l_sum * weight;
      shift = ref;
    }
    if (__all_sync(0xffffffffu, *abort_flag == 0)) {
      const float inv = l_sum > 0.f ? 1.0f / l_sum : (l_sum == 0.f ? 0.f : l_sum);    // (NaN stays NaN)
      const int64_t out = static_cast<int64_t>(item) * 128 * NT + r - r0;
      if (valid && (NT == 2 || t == 0)) p.Lpart[out] = l_sum == 0.f ? -INFINITY : (fast_log2(l_sum) - shift) * kLn2;
      const float down0 = inverse_power(up[0]) * weight, down1 = inverse_power(up[GV - 1]) * weight;
      // 32 dims at a time over this tile's Q (NT = 1: stream 1's over the pages), then
      // whole lines out of there.
      uint8_t* mine_at = smem + (NT == 2 || t == 0 ? C::kOffQ + t * C::kQTile : C::kOffRaw) + quad * 4096;
#pragma unroll 1
      for (int c = c0; c < c1; c += 32) {
        uint32_t o[32];
        tmem_ld32_nowait(tO + c, o);
        tmem_wait_ld32(o);
        const float mul = c < 64 ? down0 : down1;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float x = __uint_as_float(o[i]) * mul;
          if (NT == 1) x = fmaf(theirs[(c + i) * 128 + row], other, mine > 0 ? x : 0.f);
          o[i] = __float_as_uint(x * inv);
        }
#pragma unroll
        for (int i = 0; i < 32; i += 8) {                  // columns (0, 4, 1, 5, 2, 6, 3, 7) of eight
          uint4* to = reinterpret_cast<uint4*>(mine_at + lane * 128);
          to[(i / 4) ^ (lane & 7)] = make_uint4(o[i], o[i + 2], o[i + 4], o[i + 6]);
          to[(i / 4 + 1) ^ (lane & 7)] = make_uint4(o[i + 1], o[i + 3], o[i + 5], o[i + 7]);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int at = i * 4 + static_cast<int>(lane >> 3), chunk = static_cast<int>(lane & 7);
          const int rr = static_cast<int>(quad) * 32 + at;
          const uint4 x = *reinterpret_cast<const uint4*>(mine_at + at * 128 + (chunk ^ (at & 7)) * 16);
          if (tile0 + rr < R)
            *reinterpret_cast<uint4*>(p.Opart + (static_cast<int64_t>(item) * 128 * NT + tile0 - r0 + rr) * DV + c +
                                      4 * chunk) = x;
        }
        __syncwarp();
      }
    }
    tc_fence_before_sync();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag == 1) record_status(p.status, ATTN_ERR_TIMEOUT);
  // The sequences' own keys, whose kernel may still run, are the merge's too: it
  // waits for this grid alone.
  cudaGridDependencySynchronize();
}

template <int DH, int DV, int NT>
cudaError_t launch_t(const PrefixTileParams& p, cudaStream_t stream) {
  using C = TileCfg<DH, DV, NT>;
  auto kern = prefix_tile_kernel<DH, DV, NT>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(kern), C::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.Hkv * p.row_blocks * p.splits));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int DH, int DV>
cudaError_t launch_rows(const PrefixTileParams& p, cudaStream_t stream) {
  return p.row_tiles == 2 ? launch_t<DH, DV, 2>(p, stream) : launch_t<DH, DV, 1>(p, stream);
}

}  // namespace

cudaError_t launch_prefix_tile(int dh, int dv, const PrefixTileParams& p, cudaStream_t stream) {
  if (dh == 128 && dv == 128) return launch_rows<128, 128>(p, stream);
  if (dh == 64 && dv == 64) return launch_rows<64, 64>(p, stream);
  if (dh == 128 && dv == 64) return launch_rows<128, 64>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace esd
