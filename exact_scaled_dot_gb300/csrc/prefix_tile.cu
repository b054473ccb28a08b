// prefix_tile.cu -- the keys that a whole batch shares, for the query rows of
// all its sequences: the first part of attn_fwd_prefix_cache (prefix_cache.cu) where
// there are enough rows for the tensor core's 128-row tiles, on sm_103a.
//
// With rows = (sequences) x (query heads of a KV head) x n_q the prefix costs
// 2 rows (d_h + d_v) operations per key and head for 0.5625 (d_h + d_v) bytes:
// from a few hundred rows on it is bound by the tensor core, not by memory.  A
// CTA takes a range of the prefix for one KV head and up to 256 rows, and turns
// every tile of 64 keys (two pages) into fp16 operands once for all of them:
//
//   S_g = Q_g (c - z)_g^T   for each group g of 64 dims, exact products (c - z
//     is a small integer, Q a bf16 number times a power of two), fp32 sums
//   s_ij = f_i sum_g sk_gj S_g,ij  in fp32: the keys' scales stay out of the
//     operands, where their product with c - z would not fit fp16
//   O_g += W_g (c - z)_g,  W_g,ij = fp16(P_ij sv_gj / top_gi)
//
// with the weights' powers of two `top` per row and group as in the attention
// of a few rows over this cache (decode_cache_kernel.cuh, where they are
// explained); the zero points are in the operands here, so that O's sums need
// no correction.
//
// CTA: 512 threads, one per SM.  Warp 0 brings pages into a ring (bulk copies),
// warps 12-15 turn them into K-major and MN-major operand tiles (128-byte
// swizzle), warp 1 issues the products, warps 4-7 and 8-11 are two softmax
// streams (thread = row).  With two row tiles (NT = 2) stream t has tile t and
// both use every key tile; with one (NT = 1) the streams take the key tiles in
// turn, each with accumulators of its own, merged at the end.  While one
// stream's softmax runs, the tensor core works for the other.
//
// Tensor memory, stream t: S_0, S_1 in columns [128 t, 128 t + 128), the fp16
// weights W_0, W_1 over its first 64 once the scores are read; O in
// [256 + 128 t, + d_v).
//
// A 32-bit word of codes becomes four pairs of operands by one AND-OR and one
// fp16 operation each (0x6400 | c is 1024 + c); the pairs are the dims (k, k + 4)
// of eight, an order that Q's rows are given too and that O's columns lose again
// when they are written.
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
constexpr int kKeys = 64;           // keys of a tile: two pages
constexpr int kTilePages = kKeys / kPageTokens;

template <int DH, int DV, int NT>
struct TileCfg {
  static constexpr int GK = DH / kQuantGroup, GV = DV / kQuantGroup;
  static constexpr int kBlock = page_head_bytes(DH, DV);
  static constexpr int kRawStages = 6, kStages = NT == 2 ? 3 : 4;
  static constexpr int kQTile = 128 * DH * 2;
  static constexpr int kK16 = kKeys * DH * 2, kV16 = kKeys * DV * 2;
  static constexpr int kScales = (GK + GV) * kKeys * 4;      // floats
  static constexpr int kOffQ = 0;
  static constexpr int kOffOp = kOffQ + NT * kQTile;         // [stage] K16, V16
  static constexpr int kOffRaw = kOffOp + kStages * (kK16 + kV16);
  static constexpr int kOffScale = kOffRaw + kRawStages * kTilePages * kBlock;   // [stage] K's, V's
  static constexpr int kOffMax = kOffScale + kStages * kScales;                  // [stage][GV][2]
  static constexpr int kOffRawMask = kOffMax + kStages * 16;                     // [raw stage][2]
  static constexpr int kOffMask = kOffRawMask + kRawStages * 8;                  // [stage][2]
  static constexpr int kOffState = kOffMask + kStages * 8;   // [128] (l, shift) of stream 1 (NT = 1)
  static constexpr int kOffBar = kOffState + 128 * 8;
  static constexpr int kBarRawFull = 0;
  static constexpr int kBarRawEmpty = kBarRawFull + kRawStages;
  static constexpr int kBarFull = kBarRawEmpty + kRawStages;
  static constexpr int kBarEmpty = kBarFull + kStages;
  static constexpr int kBarS = kBarEmpty + kStages;          // [2]
  static constexpr int kBarP = kBarS + 2;                    // [2]
  static constexpr int kBarPV = kBarP + 2;                   // [2]
  static constexpr int kBarQ = kBarPV + 2;
  static constexpr int kBarDrain = kBarQ + 1;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr int kOffTmem = kOffBar + kNumBars * 8;
  static constexpr int kOffAbort = kOffTmem + 4;
  static constexpr int kSmemBytes = kOffAbort + 4 + 1024;    // slack for 1024-byte alignment
  static constexpr int kThreads = 512;
  // Registers: 128 a thread at launch, moved between the four warpgroups.
  static constexpr uint32_t kRegsLaunch = 128, kRegsControl = 64, kRegsSoftmax = 176, kRegsOperands = 96;
  static_assert(kRegsControl + 2 * kRegsSoftmax + kRegsOperands <= 4 * kRegsLaunch, "the block's registers");
  static_assert(kSmemBytes <= 232448, "shared memory");
  static_assert(kBlock % 16 == 0 && kOffRaw % 16 == 0 && kOffScale % 16 == 0 && kOffBar % 8 == 0, "alignment");
  static_assert(NT == 2 || 128 * DV * 4 <= kStages * (kK16 + kV16), "stream 1's sums over the operand tiles");
};

// The pairs (k, k + 4) of eight codes less their zero point, as fp16.
__device__ __forceinline__ uint4 operand8(uint32_t codes, uint32_t word) {
  const uint32_t z = __byte_perm(word, 0x64646464u, 0x4040);            // 1024 + z, twice
  const uint32_t z16 = ((z & 0x00FF00FFu) << 4) + 0xD400D400u;          // -(64 + z)
  auto low = [&](uint32_t x) {                                          // 1024 + c less 1024 + z
    const uint32_t v = (x & 0x000F000Fu) | 0x64006400u;
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&z));
    return *reinterpret_cast<const uint32_t*>(&r);
  };
  auto high = [&](uint32_t x) {                                         // (1024 + 16 c) / 16 - (64 + z)
    return hfma2_bits((x & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, z16);
  };
  return make_uint4(low(codes), high(codes), low(codes >> 8), high(codes >> 8));
}

template <int DH, int DV, int NT>
__global__ void __launch_bounds__(512, 1) prefix_tile_kernel(const __grid_constant__ PrefixTileParams p) {
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
  const int tiles = (len + kKeys - 1) / kKeys;
  const int each = (tiles + p.splits - 1) / p.splits;
  if (item == 0 && threadIdx.x == 0) *p.used = each > 0 ? (tiles + each - 1) / each : 0;
  const int t0 = split * each;
  const int n = tiles - t0 < each ? tiles - t0 : each;
  if (n <= 0) return;          // (the whole CTA, before it owns anything)

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kRawStages; ++s) {
      mbar_init(bar(C::kBarRawFull + s), 1);
      mbar_init(bar(C::kBarRawEmpty + s), 128);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar(C::kBarFull + s), 128);
      mbar_init(bar(C::kBarEmpty + s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(C::kBarS + t), 1);
      mbar_init(bar(C::kBarP + t), 128);
      mbar_init(bar(C::kBarPV + t), 1);
    }
    mbar_init(bar(C::kBarQ), 128 * NT);
    mbar_init(bar(C::kBarDrain), 1);
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
            const int page = (t0 + j) * kTilePages + i, left = len - page * kPageTokens;
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
    } else if (warp == 1) {
      // ================= products =================
      if (__all_sync(0xffffffffu, *abort_flag == 0)) {
        constexpr uint32_t kIdQK = idesc_f16_f32(128, kKeys, false, false);
        constexpr uint32_t kIdPV = idesc_f16_f32(128, 64, false, true);
        const SmemDesc dq0 = sw128_desc_words(sbase + C::kOffQ, 16, 1024);
        const SmemDesc dk0 = sw128_desc_words(sbase + C::kOffOp, 16, 1024);
        const SmemDesc dv0 = sw128_desc_words(sbase + C::kOffOp + C::kK16, 16, 1024);
        auto scores = [&](int t, int k) {         // S_g of stream t's k-th tile
          const SmemDesc dk = desc_step(dk0, tile_of(t, k) % C::kStages * (C::kK16 + C::kV16));
          const SmemDesc dq = desc_step(dq0, (NT == 2 ? t : 0) * C::kQTile);
#pragma unroll
          for (int g = 0; g < GK; ++g)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_ss_we(tmem + 128 * t + 64 * g, desc_step(dq, g * 128 * 128 + kk * 32),
                         desc_step(dk, g * kKeys * 128 + kk * 32), kIdQK, kk > 0 ? 1u : 0u);
          umma_commit_we(bar(C::kBarS + t));
        };
        bool ok = wait_all(C::kBarQ, 0);
        for (int t = 0; t < 2 && ok; ++t) {
          if (count_of(t) == 0) continue;
          ok = wait_all(C::kBarFull + tile_of(t, 0) % C::kStages, phase(tile_of(t, 0), C::kStages));
          if (!ok) break;
          tc_fence_after_sync();
          scores(t, 0);
        }
        for (int k = 0; k < count_of(0) && ok; ++k) {
          for (int t = 0; t < 2 && ok; ++t) {
            if (k >= count_of(t)) continue;
            ok = wait_all(C::kBarP + t, static_cast<uint32_t>(k & 1));
            if (!ok) break;
            tc_fence_after_sync();
            const int st = tile_of(t, k) % C::kStages;
            const SmemDesc dv = desc_step(dv0, st * (C::kK16 + C::kV16));
#pragma unroll
            for (int g = 0; g < GV; ++g)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_ts_we(tmem + 256 + 128 * t + 64 * g, tmem + 128 * t + 32 * g + kk * 8,
                           desc_step(dv, g * kKeys * 128 + kk * 2048), kIdPV, (k > 0 || kk > 0) ? 1u : 0u);
            umma_commit_we(bar(C::kBarPV + t));
            if (NT == 1 || t == 1) umma_commit_we(bar(C::kBarEmpty + st));
            if (k + 1 < count_of(t)) {
              const int next = tile_of(t, k + 1);
              ok = wait_all(C::kBarFull + next % C::kStages, phase(next, C::kStages));
              if (!ok) break;
              tc_fence_after_sync();
              scores(t, k + 1);
            }
          }
        }
        int no_abort = 0;
        umma_commit_we(bar(C::kBarDrain));
        mbar_wait(bar(C::kBarDrain), 0, &no_abort, limit);
      }
      __syncwarp();
    }
  } else if (warp >= 12) {
    // ================= codes into operands =================
    setmaxnreg_to<C::kRegsOperands, C::kRegsLaunch>();
    const int tid = static_cast<int>(threadIdx.x) - 384, w4 = static_cast<int>(warp) - 12;
    bool ok = *abort_flag == 0;
    for (int j = 0; j < n && ok; ++j) {
      const int rs = j % C::kRawStages, st = j % C::kStages;
      ok = wait_all(C::kBarRawFull + rs, phase(j, C::kRawStages));
      if (ok && j >= C::kStages) ok = wait_all(C::kBarEmpty + st, phase(j - C::kStages, C::kStages));
      if (!ok) break;
      const uint8_t* raw = smem + C::kOffRaw + rs * kTilePages * C::kBlock;
      uint8_t* k16 = smem + C::kOffOp + st * (C::kK16 + C::kV16);
      // A row of D dims is D / 8 words; a warp takes 256 / D rows at a time.
      auto convert = [&](auto width, int codes_at, int words_at, uint8_t* out) {
        constexpr int D = decltype(width)::value, kWords = D / 8, kRows = 32 / kWords, G = D / kQuantGroup;
        const int c = static_cast<int>(lane) % kWords;
#pragma unroll
        for (int i = 0; i < kKeys / (4 * kRows); ++i) {
          const int key = (i * 4 + w4) * kRows + static_cast<int>(lane) / kWords;
          const uint8_t* blk = raw + key / kPageTokens * C::kBlock;
          const int at = key % kPageTokens;
          const uint32_t codes = *reinterpret_cast<const uint32_t*>(blk + codes_at + at * (D / 2) + 4 * c);
          const uint32_t word = *reinterpret_cast<const uint32_t*>(blk + words_at + (at * G + c / 8) * 4);
          *reinterpret_cast<uint4*>(out + c / 8 * (kKeys * 128) + key * 128 + (((c & 7) ^ (key & 7)) * 16)) =
              operand8(codes, word);
        }
      };
      convert(std::integral_constant<int, DH>{}, off_k_codes(), off_k_words(DH, DV), k16);
      convert(std::integral_constant<int, DV>{}, off_v_codes(DH), off_v_words(DH, DV), k16 + C::kK16);
      // The keys' scales as fp32 (0 for keys that are not there), and the
      // largest of V's in each page.
      const uint32_t* masks = reinterpret_cast<const uint32_t*>(smem + C::kOffRawMask) + 2 * rs;
      float* scales = reinterpret_cast<float*>(smem + C::kOffScale + st * C::kScales);
#pragma unroll
      for (int i = 0; i < (GK + GV) * kKeys / 128 + ((GK + GV) * kKeys % 128 != 0); ++i) {
        const int at = i * 128 + tid, which = at / kKeys, key = at % kKeys;     // (a warp: one `which`, one page)
        if (which < GK + GV) {
          const int page = key / kPageTokens;
          const uint8_t* words = raw + page * C::kBlock + (which < GK ? off_k_words(DH, DV) : off_v_words(DH, DV));
          const int of = which < GK ? (key % kPageTokens) * GK + which : (key % kPageTokens) * GV + which - GK;
          const bool there = (masks[page] >> (key % kPageTokens)) & 1u;
          const uint32_t bits = there ? reinterpret_cast<const uint32_t*>(words)[of] & 0xFFFF0000u : 0u;
          scales[which * kKeys + key] = __uint_as_float(bits);
          const uint32_t most = __reduce_max_sync(0xffffffffu, bits);
          if (which >= GK && lane == 0)
            reinterpret_cast<uint32_t*>(smem + C::kOffMax)[st * 4 + (which - GK) * 2 + page] = most;
        }
      }
      if (tid < 2) (reinterpret_cast<uint32_t*>(smem + C::kOffMask) + 2 * st)[tid] = masks[tid];
      fence_proxy_async_smem();
      mbar_arrive(bar(C::kBarFull + st));
      mbar_arrive(bar(C::kBarRawEmpty + rs));
    }
  } else {
    // ================= softmax =================
    setmaxnreg_to<C::kRegsSoftmax, C::kRegsLaunch>();
    const int t = static_cast<int>(warp) / 4 - 1;          // stream
    const uint32_t quad = warp & 3;
    const int row = static_cast<int>(quad * 32 + lane), r = r0 + (NT == 2 ? 128 * t : 0) + row;
    const bool valid = r < R;
    const uint32_t lane_base = (quad * 32u) << 16;
    const uint32_t tS = tmem + lane_base + 128 * t, tO = tmem + lane_base + 256 + 128 * t;
    // ---- the row of Q: its power of two, its fp16 operands ----
    float f;
    {
      const int of = valid ? r / p.per : 0;
      const int64_t q_row = (static_cast<int64_t>(of) * p.Hkv + h) * p.per + (valid ? r - of * p.per : 0);
      const uint4* q = reinterpret_cast<const uint4*>(p.Q) + q_row * (DH / 8);
      uint4 v[DH / 8];
      uint32_t m = 0u;
#pragma unroll
      for (int c = 0; c < DH / 8; ++c) {
        v[c] = valid ? q[c] : make_uint4(0u, 0u, 0u, 0u);
        m = bf16_absmax_fold(m, v[c]);
      }
      const float mx = bf16_absmax_value(m);
      int e = 0;                                           // 2^14 <= mx 2^e < 2^15
      if (mx > 0.f && mx < INFINITY) e = 14 - ilogbf(mx);
      e = e > 120 ? 120 : e;
      // (Not 0, which a masked -inf must not meet; NaN for a row that is not finite.)
      f = fmaxf(p.scale_log2 * exp2_int(-e), 0x1p-126f);
      if (!(mx < INFINITY)) f = __uint_as_float(0x7FC00000u);
      if (NT == 2 || t == 0) {
        uint8_t* to = smem + C::kOffQ + (NT == 2 ? t : 0) * C::kQTile + row * 128;
#pragma unroll
        for (int c = 0; c < DH / 8; ++c) {
          const uint4 u = bf16x8_to_f16x8_scaled(v[c], exp2_int(e));
          *reinterpret_cast<uint4*>(to + c / 8 * (128 * 128) + (((c & 7) ^ (row & 7)) * 16)) =
              make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632), __byte_perm(u.y, u.w, 0x5410),
                         __byte_perm(u.y, u.w, 0x7632));
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(C::kBarQ));
      }
    }
    float shift = -kNoKey, l_sum = 0.f;        // less the reference that P is relative to; the sum of P
    float up[GV], s_lim[GV];                   // 1 / top; the scale from which on a weight may be too large
#pragma unroll
    for (int g = 0; g < GV; ++g) up[g] = exp2_int(-kLeastTop), s_lim[g] = 0.f;
    uint32_t seen = 0u;                        // keys there were
    const int mine = count_of(t);
    bool ok = *abort_flag == 0;
    for (int k = 0; k < mine && ok; ++k) {
      const int j = tile_of(t, k), st = j % C::kStages;
      ok = wait_all(C::kBarS + t, static_cast<uint32_t>(k & 1)) && wait_all(C::kBarFull + st, phase(j, C::kStages));
      if (!ok) break;
      tc_fence_after_sync();
      const float* scales = reinterpret_cast<const float*>(smem + C::kOffScale + st * C::kScales);
      // ---- scores ----
      float s[kKeys];
#pragma unroll
      for (int c = 0; c < kKeys / 32; ++c) {
        uint32_t a[GK][32];
#pragma unroll
        for (int g = 0; g < GK; ++g) tmem_ld32_nowait(tS + 64 * g + 32 * c, a[g]);
#pragma unroll
        for (int g = 0; g < GK; ++g) tmem_wait_ld32(a[g]);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          float* x = s + 32 * c + i;
#pragma unroll
          for (int g = 0; g < GK; ++g) {
            const float4 sk = *reinterpret_cast<const float4*>(scales + g * kKeys + 32 * c + i);
            auto at = [&](int o) { return __uint_as_float(a[g][i + o]); };
            if (g == 0) {
              fmul2(x[0], x[1], at(0), at(1), sk.x, sk.y);
              fmul2(x[2], x[3], at(2), at(3), sk.z, sk.w);
            } else {
              ffma2(x[0], x[1], at(0), at(1), sk.x, sk.y, x[0], x[1]);
              ffma2(x[2], x[3], at(2), at(3), sk.z, sk.w, x[2], x[3]);
            }
          }
        }
      }
      const uint2 mask = *reinterpret_cast<const uint2*>(smem + C::kOffMask + 8 * st);
      seen |= mask.x | mask.y;
      if ((mask.x & mask.y) != 0xFFFFFFFFu) {
#pragma unroll
        for (int i = 0; i < kKeys; ++i)
          if (!(((i < 32 ? mask.x : mask.y) >> (i & 31)) & 1u)) s[i] = -INFINITY;
      }
      // ---- running maximum (lazy) and the weights' scales ----
      float mx = fmaxf(s[0], s[1]), mx2 = fmaxf(s[2], s[3]);
#pragma unroll
      for (int i = 4; i < kKeys; i += 4) {
        mx = fmax3(mx, s[i], s[i + 1]);
        mx2 = fmax3(mx2, s[i + 2], s[i + 3]);
      }
      mx = fmaxf(mx, mx2);
      bool need = fmaf(mx, f, shift) > static_cast<float>(kLazy);
#pragma unroll
      for (int g = 0; g < GV; ++g) {
        const float2 sm = *reinterpret_cast<const float2*>(smem + C::kOffMax + st * 16 + g * 8);
        need |= fmaxf(sm.x, sm.y) > s_lim[g];
      }
      const float* sv = scales + GK * kKeys;
      if (__any_sync(0xffffffffu, need)) {
        const float m = ceilf(mx * f);
        float alpha = 1.f;
        if (m + shift > static_cast<float>(kLazy)) {       // (whole octaves: alpha is a power of two)
          alpha = fast_exp2(-shift - m);
          shift = -m;
        }
        l_sum *= alpha;
        float most[GV], back[GV];
        bool change = false;
#pragma unroll
        for (int g = 0; g < GV; ++g) most[g] = 0.f;
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
          const float w = fast_exp2(fmaf(s[i], f, shift));
#pragma unroll
          for (int g = 0; g < GV; ++g) most[g] = fmaxf(most[g], w * sv[g * kKeys + i]);
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
          ok = wait_all(C::kBarPV + t, static_cast<uint32_t>((k - 1) & 1));
          if (!ok) break;
          tc_fence_after_sync();
#pragma unroll
          for (int g = 0; g < GV; ++g)
#pragma unroll
            for (int c = 0; c < 64; c += 16) {
              uint32_t o[16];
              tmem_ld16_nowait(tO + 64 * g + c, o);
              tmem_wait_ld16(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * back[g]);
              tmem_st16_nowait(tO + 64 * g + c, o);
            }
        }
      }
      // ---- weights ----
#pragma unroll
      for (int c = 0; c < kKeys; c += 32) {
        uint32_t w[GV][16];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          float e[4];
          const float* x = s + c + i;
          ffma2(e[0], e[1], x[0], x[1], f, f, shift, shift);
          ffma2(e[2], e[3], x[2], x[3], f, f, shift, shift);
#pragma unroll
          for (int u = 0; u < 4; ++u) e[u] = fast_exp2(e[u]);
          l_sum += (e[0] + e[1]) + (e[2] + e[3]);
#pragma unroll
          for (int g = 0; g < GV; ++g) {
            const float4 sc = *reinterpret_cast<const float4*>(sv + g * kKeys + c + i);
            float y[4];
            fmul2(y[0], y[1], e[0], e[1], up[g], up[g]);
            fmul2(y[2], y[3], e[2], e[3], up[g], up[g]);
            fmul2(y[0], y[1], y[0], y[1], sc.x, sc.y);
            fmul2(y[2], y[3], y[2], y[3], sc.z, sc.w);
            w[g][i / 2] = pack_half2(y[0], y[1]);
            w[g][i / 2 + 1] = pack_half2(y[2], y[3]);
          }
        }
#pragma unroll
        for (int g = 0; g < GV; ++g) tmem_st16_nowait(tS + 32 * g + c / 2, w[g]);
      }
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive(bar(C::kBarP + t));
    }
    if (ok && mine > 0) ok = wait_all(C::kBarPV + t, static_cast<uint32_t>((mine - 1) & 1));
    tc_fence_after_sync();
    if (seen == 0u) l_sum = 0.f;
    float weight = 1.f, other = 0.f;           // of this stream's sums and of the other's (NT = 1)
    float* theirs = reinterpret_cast<float*>(smem + C::kOffOp);        // [dim][row], over the operand tiles
    if constexpr (NT == 1) {
      // Both streams' products are done: stream 1 hands its sums to stream 0.
      named_bar_sync(1, 256);
      float2* state = reinterpret_cast<float2*>(smem + C::kOffState);
      if (t == 1) {
        state[row] = make_float2(l_sum, shift);
        if (mine > 0) {
#pragma unroll
          for (int c = 0; c < DV; c += 16) {
            uint32_t o[16];
            tmem_ld16_nowait(tO + c, o);
            tmem_wait_ld16(o);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              theirs[(c + i) * 128 + row] = __uint_as_float(o[i]) * inverse_power(up[c / 64]);
          }
        }
      }
      named_bar_sync(1, 256);
      if (t == 0 && count_of(1) > 0) {
        const float2 x = state[row];
        const float ref = fminf(shift, x.y);   // less the larger reference
        weight = fast_exp2(ref - shift);
        other = fast_exp2(ref - x.y);
        l_sum = l_sum * weight + x.x * other;
        shift = ref;
      }
    }
    if ((NT == 2 || t == 0) && __all_sync(0xffffffffu, *abort_flag == 0)) {
      const float inv = l_sum > 0.f ? 1.0f / l_sum : (l_sum == 0.f ? 0.f : l_sum);    // (NaN stays NaN)
      const int64_t out = static_cast<int64_t>(item) * 128 * NT + r - r0;
      if (valid) p.Lpart[out] = l_sum == 0.f ? -INFINITY : (fast_log2(l_sum) - shift) * kLn2;
      float* dst = p.Opart + out * DV;
#pragma unroll
      for (int c = 0; c < DV; c += 16) {
        uint32_t o[16];
        tmem_ld16_nowait(tO + c, o);
        tmem_wait_ld16(o);
        const float mul = inverse_power(up[c / 64]) * weight;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          x[i] = __uint_as_float(o[i]) * mul;
          if (NT == 1 && count_of(1) > 0) x[i] = fmaf(theirs[(c + i) * 128 + row], other, x[i]);
          x[i] *= inv;
        }
        if (valid) {
#pragma unroll
          for (int i = 0; i < 16; i += 8) {                // columns (0, 4, 1, 5, 2, 6, 3, 7) of eight
            *reinterpret_cast<float4*>(dst + c + i) = make_float4(x[i], x[i + 2], x[i + 4], x[i + 6]);
            *reinterpret_cast<float4*>(dst + c + i + 4) = make_float4(x[i + 1], x[i + 3], x[i + 5], x[i + 7]);
          }
        }
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
}

template <int DH, int DV, int NT>
cudaError_t launch_t(const PrefixTileParams& p, cudaStream_t stream) {
  using C = TileCfg<DH, DV, NT>;
  auto kern = prefix_tile_kernel<DH, DV, NT>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(p.Hkv * p.row_blocks * p.splits), C::kThreads, C::kSmemBytes, stream>>>(p);
  return cudaGetLastError();
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
