// cache_weigh.cu -- attn_cache_weigh: the attention weight that each cached
// token gets from the new queries, added to what it has had, on sm_103a.
//
//   w[b][h][j] += sum over the query heads r of KV head h and the rows i that
//                 see key j of A_ij,  A_ij = exp(scale q_i . k_j - LSE_i)
// ("Appendix A.10 -- Attention matrices and backpropagation", eqs. A.10.1 and
// A.10.2 with the log-sum-exp of the attention, over whatever keys that had).
// The normaliser is given, so there is no running maximum and every page is on
// its own: keys are the M side of K Q^T, as in the attention over this cache,
// and a key's weight is a sum over its row of the accumulators, in one order.
//
// Work: the pages of all sequences, end to end, are cut into equal ranges, one
// per CTA of a KV head; its warps take every fourth page.  A lane's codes are what
// it needs of 16 keys as fragments, so that they go from device memory to
// registers; the warps of an SM hide one another's loads, and the page after the
// next is on its way to the second-level cache.  Q's fragments are kept in shared
// memory, a sequence at a time, so that up to 256 query rows pass over a page that
// is read once.
//
// Measured (GB300, device time).  8 sequences of 16-32 thousand keys, 32 heads on 8,
// widths 128: 36 us for 126 MB, 3.5 TB/s (its floor 18.6).  48 of 4-12000 keys, 4
// queries, 16 heads on 4, widths 128 and 64: 31 us for 93 MB (13.7).  One of 700 keys:
// 3.9.  Bound by the issue of instructions and their latencies: some 456 a page and
// head, a third of them codes into fragments, which eight rows' products then use
// once; the schedulers issue in 51 % of the cycles with four warps each (128
// registers), ALU 41, tensor pipe 18, DRAM 47 %.  (Pages by bulk copies through shared
// memory, as the attention has them: 43 and 34 us.  A page's codes requested as soon
// as the page before is fragments: 35 and 32; three CTAs an SM: 44 and 35.)
#include <cstdint>
#include <cuda_runtime.h>

#include "cache_mma.cuh"

namespace esd {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kResident = kCacheWeighResident;     // CTAs per SM that the registers are held to
constexpr int kAhead = 1;             // pages that a warp has on their way to the second-level cache
constexpr int kMostGroups = 32;       // of eight query rows in shared memory: more pass over the pages again

// What two rows of Q bring, row r and r + 1: p = exp2(f s + add) for the keys below lim.
struct __align__(16) RowTerms {
  float f[2], add[2];
};

template <int DH, int DV>
struct WeighCfg {
  static constexpr int GK = DH / kQuantGroup;
  static constexpr int kBlock = page_head_bytes(DH, DV);
  static constexpr int kCodes = kPageTokens * DH / 2, kWords = kPageTokens * GK * 4;
  // Eight query rows: their terms, their limits and, of each group of 64 dims, two
  // 16-byte chunks of fp16 fragments per lane.
  static constexpr int kLimits = 4 * static_cast<int>(sizeof(RowTerms)), kFragments = kLimits + 64;
  static constexpr int kRowBytes = kFragments + GK * 2 * 32 * 16;
  static int smem_bytes(int row_groups) { return row_groups * kRowBytes; }
};

template <int DH, int DV>
__global__ void __launch_bounds__(kThreads, kResident) cache_weigh_kernel(const __grid_constant__ CacheWeighParams p) {
  using C = WeighCfg<DH, DV>;
  constexpr int GK = C::GK;
  extern __shared__ __align__(128) uint8_t smem[];
  if (__syncthreads_or(status_blocks(p.status))) return;
  const uint32_t warp = warp_id(), lane = lane_id();
  const int g = static_cast<int>(lane >> 2), t = static_cast<int>(lane & 3);
  const Ranges rg = page_ranges(p, lane);

  const int h = static_cast<int>(blockIdx.x) / p.ranges;
  const int range = static_cast<int>(blockIdx.x) - h * p.ranges;
  const int R = p.group * p.n_q, groups = (R + 7) / 8;
  const int begin = range * rg.per;
  const int end = begin + rg.per < rg.total ? begin + rg.per : rg.total;
  int b = p.B, seq0 = 0;           // the sequence that `begin` lies in, and its first page's place
  if (begin < rg.total) b = sequence_at(p, begin, lane, seq0);

  // This head's blocks: codes and words of this lane's keys, and the line it prefetches.
  const uint32_t page_stride = static_cast<uint32_t>(p.Hkv) * C::kBlock;
  const uint8_t* const head = p.pool + static_cast<int64_t>(h) * C::kBlock;
  const uint8_t* const codes_at = head + off_k_codes() + g * (DH / 2) + t * 8;
  const uint8_t* const words_at = head + off_k_words(DH, DV) + g * (GK * 4);
  constexpr int kLines = (C::kCodes + 127) / 128;
  static_assert(kLines < 30, "a lane per line");
  const uint8_t* const line_at = static_cast<int>(lane) < kLines ? head + 128 * lane : head + off_k_words(DH, DV) + 128 * (lane - kLines);
  const bool has_line = static_cast<int>(lane) < kLines + (C::kWords + 127) / 128;
  for (; b < p.B; ++b) {
    int len;
    const int npages = pages_of(p, b, len);
    if (seq0 >= end) break;
    if (npages == 0) continue;
    const int first = begin > seq0 ? begin - seq0 : 0;
    const int last = end < seq0 + npages ? end - seq0 : npages;
    seq0 += npages;

    for (int g0 = 0; g0 < groups; g0 += kMostGroups) {
    const int g_end = groups - g0 < kMostGroups ? groups - g0 : kMostGroups;
    // This warp's pages: first + warp, + kWarps, ...
    const int mine = (last - first - static_cast<int>(warp) + kWarps - 1) / kWarps;
    const int n = mine > 0 ? mine : 0;
    const int32_t* table = p.table + static_cast<int64_t>(b) * p.max_pages + first + warp;
    // Page numbers of 32 of them, one per lane; -1 outside the pool.
    auto numbers = [&](int from) {
      const int at = from + static_cast<int>(lane);
      int id = at < n ? table[at * kWarps] : 0;
      if (id < 0 || id >= p.pages) {
        record_status(p.status, ATTN_ERR_PAGE);
        id = -1;
      }
      return id;
    };
    int ids = numbers(0), ids_next = 0;
    // Page i of this warp's, the window of 32 that `done` is in or the next.
    auto number = [&](int i, int done) {
      return __shfl_sync(0xffffffffu, ((i ^ done) & ~31) ? ids_next : ids, i & 31);
    };
    auto prefetch = [&](int id) {
      if (has_line && id >= 0)
        asm volatile("prefetch.global.L2 [%0];" :: "l"(line_at + static_cast<uint64_t>(static_cast<uint32_t>(id)) * page_stride));
    };
    // ---- Q's fragments and the rows' terms, eight rows a warp at a time ----
    // (dims of a lane as in the attention: k-step 4 gk + 2 w + e holds the dims
    // 64 gk + 16 t + 8 w + {2e, 2e+4} and {2e+1, 2e+5}.)
    for (int nt = static_cast<int>(warp); nt < g_end; nt += kWarps) {
      const int r = 8 * (g0 + nt) + g;
      const int64_t row = (static_cast<int64_t>(b) * p.Hkv + h) * R + (r < R ? r : 0);
      const uint4* q = reinterpret_cast<const uint4*>(p.Q) + row * (DH / 8);
      const float lse = r < R ? p.LSE[row] : -INFINITY;
      uint4 qv[GK][2];
      uint32_t m = 0u;
#pragma unroll
      for (int gk = 0; gk < GK; ++gk)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          qv[gk][w] = r < R ? q[gk * 8 + 2 * t + w] : make_uint4(0u, 0u, 0u, 0u);
          // (Adds nothing, whatever it holds: a NaN would pass the -inf below.)
          if (lse == -INFINITY) qv[gk][w] = make_uint4(0u, 0u, 0u, 0u);
          m = bf16_absmax_fold(m, qv[gk][w]);
        }
      uint32_t mb = __float_as_uint(bf16_absmax_value(m));     // (as bits, so that a NaN is the largest)
      mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
      mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
      const float mx = __uint_as_float(mb);
      int e = 0;                                               // 2^14 <= mx 2^e < 2^15
      if (mx > 0.f && mx < INFINITY) e = 14 - ilogbf(mx);
      e = e > 120 ? 120 : e;
      uint8_t* to = smem + nt * C::kRowBytes;
      uint4* frag = reinterpret_cast<uint4*>(to + C::kFragments) + lane;
#pragma unroll
      for (int gk = 0; gk < GK; ++gk)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint4 u = bf16x8_to_f16x8_scaled(qv[gk][w], exp2_int(e));
          frag[(gk * 2 + w) * 32] = make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632),
                                               __byte_perm(u.y, u.w, 0x5410), __byte_perm(u.y, u.w, 0x7632));
        }
      if (t == 0) {
        float fac = fmaxf(p.scale_log2 * exp2_int(-e) * 512.0f, 0x1p-126f);
        if (!(mx < INFINITY)) fac = __uint_as_float(0x7FC00000u);
        const int lim = r < R ? len - p.n_q + 1 + r % p.n_q : 0;
        float add = -lse * kLog2e;
        // Rows without a key, and none at all, add nothing.
        if (lim <= 0 || lse == -INFINITY) fac = 0x1p-126f, add = -INFINITY;
        RowTerms& x = reinterpret_cast<RowTerms*>(to)[g >> 1];
        x.f[g & 1] = fac;
        x.add[g & 1] = add;
        reinterpret_cast<int*>(to + C::kLimits)[g] = lim;
      }
    }
    for (int i = 0; i < kAhead && i < n; ++i) prefetch(number(i, 0));
    __syncthreads();

    float* const wrow = p.weights + (static_cast<int64_t>(b) * p.Hkv + h) * p.max_pages * kPageTokens;
    for (int done = 0; done < n; ++done) {
      const int key0 = (first + static_cast<int>(warp) + done * kWarps) * kPageTokens;
      if ((done & 31) == 0) {
        if (done > 0) ids = ids_next;
        if (done + 32 < n) ids_next = numbers(done + 32);
      }
      const int id = number(done, done);
      if (done + kAhead < n) prefetch(number(done + kAhead, done));
      if (id < 0) continue;
      const uint64_t page = static_cast<uint64_t>(static_cast<uint32_t>(id)) * page_stride;
      // ---- this lane's codes and words: keys 8 i + g ----
      uint2 codes[4][GK];
      uint32_t words[4][GK];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int gk = 0; gk < GK; ++gk)
          codes[i][gk] = __ldg(reinterpret_cast<const uint2*>(codes_at + page + 8 * i * (DH / 2) + gk * 32));
        if constexpr (GK == 2) {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(words_at + page + 8 * i * 8));
          words[i][0] = w.x, words[i][1] = w.y;
        } else {
          words[i][0] = __ldg(reinterpret_cast<const uint32_t*>(words_at + page + 8 * i * 4));
        }
      }
      // The key that the page's sums over rows end with in this lane.
      const int key = key0 + 8 * t + g;
      const bool mine_here = key < len;
      const float was = mine_here ? wrow[key] : 0.f;
      const bool edge = key0 + kPageTokens > len - p.n_q + 1;   // some row does not see all of the page
      float sum[4] = {0.f, 0.f, 0.f, 0.f};                      // of the lane's rows: keys 8 i + g
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        // ---- 16 keys' codes as fragments, (c - z) 2^-9 ----
        uint32_t a[GK][4][4];
        float sa[GK], sb[GK];
        const uint32_t(&pa)[GK] = words[2 * kb], (&pb)[GK] = words[2 * kb + 1];
#pragma unroll
        for (int gk = 0; gk < GK; ++gk) {
          const uint2 wa = codes[2 * kb][gk], wb = codes[2 * kb + 1][gk];
          const uint32_t za = hfma2_bits(__byte_perm(pa[gk], 0u, 0x4040), kMinusTwo15, 0u);
          const uint32_t zb = hfma2_bits(__byte_perm(pb[gk], 0u, 0x4040), kMinusTwo15, 0u);
#pragma unroll
          for (int step = 0; step < 4; ++step) {
            uint32_t xa = step < 2 ? wa.x : wa.y, xb = step < 2 ? wb.x : wb.y;
            if (step & 1) xa >>= 8, xb >>= 8;
            a[gk][step][0] = hfma2_bits(low_nibbles(xa), kTwo15, za);
            a[gk][step][1] = hfma2_bits(low_nibbles(xb), kTwo15, zb);
            a[gk][step][2] = hfma2_bits(high_nibbles(xa), kTwo11, za);
            a[gk][step][3] = hfma2_bits(high_nibbles(xb), kTwo11, zb);
          }
          sa[gk] = bf16_hi(pa[gk]);
          sb[gk] = bf16_hi(pb[gk]);
        }
        // ---- the sums over all rows, eight at a time ----
        float s0 = 0.f, s1 = 0.f;
        for (int nt = 0; nt < g_end; ++nt) {
          const uint8_t* from = smem + nt * C::kRowBytes;
          const uint4* frag = reinterpret_cast<const uint4*>(from + C::kFragments) + lane;
          const float4 x = *reinterpret_cast<const float4*>(from + t * sizeof(RowTerms));
          float s[4];
#pragma unroll
          for (int gk = 0; gk < GK; ++gk) {
            const uint4 q0 = frag[gk * 64], q1 = frag[gk * 64 + 32];
            float acc[4];
            const uint32_t(*k)[4] = a[gk];
            mma_f16(acc, k[0][0], k[0][1], k[0][2], k[0][3], q0.x, q0.y, 0.f, 0.f, 0.f, 0.f);
            mma_f16(acc, k[1][0], k[1][1], k[1][2], k[1][3], q0.z, q0.w);
            mma_f16(acc, k[2][0], k[2][1], k[2][2], k[2][3], q1.x, q1.y);
            mma_f16(acc, k[3][0], k[3][1], k[3][2], k[3][3], q1.z, q1.w);
            if (gk == 0) {
              fmul2(s[0], s[1], acc[0], acc[1], sa[gk], sa[gk]);
              fmul2(s[2], s[3], acc[2], acc[3], sb[gk], sb[gk]);
            } else {
              ffma2(s[0], s[1], acc[0], acc[1], sa[gk], sa[gk], s[0], s[1]);
              ffma2(s[2], s[3], acc[2], acc[3], sb[gk], sb[gk], s[2], s[3]);
            }
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float p0, p1;
            ffma2(p0, p1, s[2 * i], s[2 * i + 1], x.x, x.y, x.z, x.w);
            p0 = fast_exp2(p0);
            p1 = fast_exp2(p1);
            if (edge) {
              const int k = key0 + 16 * kb + 8 * i + g;
              const int2 lim = reinterpret_cast<const int2*>(from + C::kLimits)[t];
              p0 = k < lim.x ? p0 : 0.f;
              p1 = k < lim.y ? p1 : 0.f;
            }
            (i == 0 ? s0 : s1) += p0 + p1;
          }
        }
        sum[2 * kb] = s0, sum[2 * kb + 1] = s1;
      }
      // Over the four lanes of a key; lane t ends with the keys 8 t + g.
      const float keep0 = t & 2 ? sum[2] : sum[0], keep1 = t & 2 ? sum[3] : sum[1];
      const float give0 = t & 2 ? sum[0] : sum[2], give1 = t & 2 ? sum[1] : sum[3];
      const float two0 = keep0 + __shfl_xor_sync(0xffffffffu, give0, 2);
      const float two1 = keep1 + __shfl_xor_sync(0xffffffffu, give1, 2);
      const float all = (t & 1 ? two1 : two0) + __shfl_xor_sync(0xffffffffu, t & 1 ? two0 : two1, 1);
      if (mine_here) wrow[key] = was + all;
    }
    __syncthreads();           // the rows' fragments are free for the next ones
    }
  }
}

template <int DH, int DV>
cudaError_t launch_t(const CacheWeighParams& p, cudaStream_t stream) {
  using C = WeighCfg<DH, DV>;
  const int groups = (p.group * p.n_q + 7) / 8;
  const int bytes = C::smem_bytes(groups < kMostGroups ? groups : kMostGroups);
  auto kern = cache_weigh_kernel<DH, DV>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(kern), C::smem_bytes(kMostGroups), done);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(p.Hkv * p.ranges), kThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_weigh(int dh, const CacheWeighParams& p, int dv, cudaStream_t stream) {
  if (dh == 128 && dv == 128) return launch_t<128, 128>(p, stream);
  if (dh == 64 && dv == 64) return launch_t<64, 64>(p, stream);
  if (dh == 128 && dv == 64) return launch_t<128, 64>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace esd
