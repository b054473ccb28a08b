// decode_cache.cu -- forward attention of a few new queries per sequence over
// the paged 4-bit key/value cache (quant_cache.cuh), on sm_103a.
//
// Same function as the decode forward ("Appendix A.10 -- Attention matrices
// and backpropagation", eqs. A.10.1-A.10.3; the new-queries-over-a-history
// shape of "Chapter 31 -- attention backprop", section 1) with
// K_j = s (code - z) and V_j likewise: row i of n_q sees the keys
// j <= len - n_q + i.
//
// The cache is read once per KV head, 0.5625 bytes per element, which bounds
// the call; the codes must become matrix operands at that pace (some 40
// elements per SM and cycle).  So they stay in registers between shared
// memory and the tensor core, as fragments of mma.sync (through shared
// memory, tcgen05's operands would cost a 2-byte write and read per element,
// several times the traffic of the codes; through tensor memory, its A operand
// would: not measured), with the cache as the M side of
// both products and the R = group n_q query rows of a KV head as N = 8 NT
// columns:
//   S^T = K Q^T: A = 16 keys x 16 dims.  A lane's nibbles of one key are its
//     A registers; which dims a lane holds is free as long as Q's fragments
//     agree.  code - z is exact in fp16 and Q is scaled to fp16 by a power of
//     two (exact, f16range.cuh's argument); the group's scale multiplies the
//     fp32 sums.
//   O^T = V^T P^T: A = 16 dims x 16 keys of codes; the scale goes into the
//     weights, w = P s_j, so each group of 64 dims has a B of its own.  S^T's
//     accumulators, packed to fp16 and transposed 8x8 by movmatrix, are B's
//     registers.
// A code becomes fp16 by one AND: the bits 0..3 of a half-word alone are the
// subnormal c 2^-24, the bits 4..7 are 16 c 2^-24.  For V that is the operand:
// the factor 16 is taken out of O's rows at the end, and the zero points'
// share sum_j w_ij z_j is summed in fp32 beside it, from the rounded weights
// (as a 17th row of the product it cost 8 % more time).  For K an fma makes it
// (c - z) 2^-9: the tensor core aligns a subnormal's product as if it were
// 2^-14, which costs the sums 4 to 5 bits (measured: LSE off by 8e-6 instead of
// 3e-7), too many for the scores and none that matter for O.  But it also cuts
// a sum by up to 2^-23 at every step, always downwards, and the sums of codes
// grow with the keys where O, of values around 0, does not.  So every 32 pages
// the zero points' share is taken out of O's accumulators (2-norm of the error of
// 64 sequences of 32768 keys 0.0033 without, 0.0018 with it, bf16's own; of 320000
// keys in one CTA 0.089 and 0.0019; 101.2 and 102.0 us for the first case below).
//
// fp16 weights: w = P s_j / top, with a power of two top for each query row and
// group of 64 dims that leaves the largest P s_j the row has met at 2^5 to 2^6.
// A large scale on a key that a row hardly weighs, in another group or under a
// mask takes no bits from the row's other weights, and top falls with P when the
// row's reference moves.  Both are set anew, and O rescaled, only when a score
// passes the reference by 2^5 or the page has a scale that might take a weight
// past fp16 (from 16 to 32 times the weighted one behind top on); P s_j of the page
// is formed for that in fp32.  Weights down to 2^-19 of the row's largest keep 11
// bits, smaller ones are rounded to multiples of 2^-29 of it.  Sums, maxima and O
// are fp32, and the sum of the P carries no scale of the values: it cannot leave
// fp32's range, and the LSE does not depend on V.  (One exponent for a warp, above
// every scale it had met, lost the weights beside a scale 2^24 times theirs; the
// cases below took 0.5 % less with it.  Scales spread over 16 octaves from key to
// key set top in every page: 52.2 us for the long case below instead of 49.8, 48.9
// for the ragged one instead of 44.4; over 4 octaves 50.2 and 45.1, some 10 % more
// for the ragged one with 2^7 and 4 in place of 2^5 and 16.)
//
// Work: for one (KV head, row tile), short sequences get a CTA each.  Else the
// pages of all sequences, one after the other, are cut into equal ranges, one
// per CTA (the lengths are on the device, so each CTA finds its range from
// them), and the CTAs of all tiles are resident at once: no CTA waits for a
// place, and ragged lengths cost nothing.  A CTA's warps take every fourth
// (eighth) page of a sequence, each with a ring of pages of its own (one bulk
// copy per page) and its own softmax state, and merge at the sequence's end.
// A sequence that lies in one range is written out directly; the others'
// parts are joined by the merge kernel by their log-sum-exp, as in the decode
// forward.  (attn_api.cu's plan has the rule and what both measured.)
//
// Measured (GB300, device time).  256 sequences of 2048 keys, 32 query heads on
// 8, widths 128: 102 us for 604 MB, 5.9 TB/s.  Eight of 16-32 thousand keys:
// 50 us, of which the merge 4; the 248 MB take 37 us at the measured copy rate,
// and the kernel without its arithmetic 43.  48 sequences of 4-12000 keys, 4
// queries, 16 heads on 4, widths 128 and 64: 44.5 us for 125 MB (19 us).  No unit
// is full: in these two the schedulers issue in 0.59 and 0.52 of the cycles (some
// 590 instructions a page), the ALUs are at 52 and 38 %, the tensor pipe at 28 and
// 34.  The registers (128 and 168 a thread) leave 3.7 and 2.8 warps a scheduler,
// and these wait for the fixed latencies of a page's chains (1.4 and 1.5 cycles an
// issue), for one another (not selected 1.1 and 0.7, math pipe 0.8 and 0.6,
// dispatch 0.5 and 0.4) and for pages (long scoreboard 0.8 and 0.4).
// More or fewer warps, a page of lookahead for the scores, pages or lengths
// requested across sequences, a deeper ring and an earlier or later start of
// the merge changed nothing or cost up to 2 % (tried and left out).
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "f16range.cuh"
#include "ptx.cuh"
#include "quant_cache.cuh"

namespace esd {
namespace {

constexpr float kNoKey = -1e30f;    // the reference (exp2 domain) of a row that has seen no key
// Weights w = P s_j / top of a row and group: up to 2^kTopBits when top is set,
// 2^kLazy more for a score above the row's reference and 2^kSlack more for a
// larger scale before either is set again.
constexpr int kLazy = 5, kSlack = 4, kTopBits = 6;
static_assert(kLazy + kSlack + kTopBits <= 15, "weights are fp16");
constexpr int kLeastTop = -118, kMostTop = 126;    // (exponents; P / top is at most 2^125)
// Pages of a warp after which the zero points' share is taken out of O's sums
// (error of the first of these cases 0.0018 with 8, 16 and 32, 0.0018 to 0.0019 with 64).
constexpr int kZeroPages = 32;
constexpr int kStages = 3;

// d = A B + c (m16n8k16, fp16 operands, fp32 sums).
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, float c0, float c1, float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  mma_f16(d, a0, a1, a2, a3, b0, b1, d[0], d[1], d[2], d[3]);
}

// The 8x8 matrix of 16-bit elements spread over the warp (lane 4r + c holds
// columns 2c, 2c+1 of row r), transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Four 8x8 matrices of 16-bit elements from shared memory, transposed: lanes
// 8j..8j + 7 address the rows of matrix j; lane 4r + c gets its elements
// (2c, r) and (2c + 1, r).
__device__ __forceinline__ void load_transposed(uint32_t row, uint32_t (&x)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(row) : "memory");
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

__device__ __forceinline__ uint2 lds64(const uint8_t* p) { return *reinterpret_cast<const uint2*>(p); }
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 2) {
    const uint2 v = lds64(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// The fp16 operands c 2^-24 of bits 0-3, and 16 c 2^-24 of bits 4-7, of both
// halves of x.
__device__ __forceinline__ uint32_t low_nibbles(uint32_t x) { return x & 0x000F000Fu; }
__device__ __forceinline__ uint32_t high_nibbles(uint32_t x) { return x & 0x00F000F0u; }

__device__ __forceinline__ uint32_t hfma2_bits(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                            *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
constexpr uint32_t kTwo15 = 0x78007800u, kTwo11 = 0x68006800u, kMinusTwo15 = 0xF800F800u;   // fp16 pairs

// acc + a b, a the lower (upper) fp16 of w and b the fp16 in the lower half of
// z, in fp32 with one rounding.
__device__ __forceinline__ void fma_halves(float& acc0, float& acc1, uint32_t w, uint32_t z) {
  asm("{\n\t.reg .b16 w0, w1, z0, z1;\n\t"
      "mov.b32 {w0, w1}, %2;\n\tmov.b32 {z0, z1}, %3;\n\t"
      "fma.rn.f32.f16 %0, w0, z0, %0;\n\tfma.rn.f32.f16 %1, w1, z0, %1;\n\t}"
      : "+f"(acc0), "+f"(acc1)
      : "r"(w), "r"(z));
}

// Powers of two: the next one from x >= 0 up (0: 0), the nearest, and 1 / x of one.
__device__ __forceinline__ uint32_t next_power(float x) { return (__float_as_uint(x) + 0x007FFFFFu) & 0x7F800000u; }
__device__ __forceinline__ uint32_t near_power(float x) { return (__float_as_uint(x) + 0x00400000u) & 0x7F800000u; }
__device__ __forceinline__ float inverse_power(float x) { return __uint_as_float(0x7F000000u - __float_as_uint(x)); }

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Pages of sequence b, its length cut to the page table's.
__device__ __forceinline__ int pages_of(const DecCacheParams& p, int b, int& len) {
  const int cap = p.max_pages * kPageTokens;
  len = p.lengths[b];
  len = len < 0 ? 0 : (len > cap ? cap : len);
  return (len + kPageTokens - 1) / kPageTokens;
}

// How the pages of all sequences, laid end to end, are cut into ranges of one
// CTA each: range i is [i per, (i + 1) per).  Called by whole warps.
struct Ranges {
  int total, per;
};
__device__ __forceinline__ Ranges page_ranges(const DecCacheParams& p, uint32_t lane) {
  int sum = 0, len;
  for (int b = static_cast<int>(lane); b < p.B; b += 32) {
    sum += pages_of(p, b, len);
    if (blockIdx.x == 0 && p.lengths[b] > p.max_pages * kPageTokens) record_status(p.status, ATTN_ERR_PAGE);
  }
  sum = __reduce_add_sync(0xffffffffu, sum);
  const int per = (sum + p.ranges - 1) / p.ranges;
  return Ranges{sum, per < kMinRangePages ? kMinRangePages : per};
}

// Pages of 32 sequences from b0 on, this lane's, and the pages up to and
// including it.
__device__ __forceinline__ int scan_pages(const DecCacheParams& p, int b0, uint32_t lane, int& incl) {
  int len;
  const int b = b0 + static_cast<int>(lane);
  const int n = b < p.B ? pages_of(p, b, len) : 0;
  incl = n;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, off);
    if (static_cast<int>(lane) >= off) incl += v;
  }
  return n;
}

template <int DH, int DV, int NT, int WARPS, bool WHOLE>
struct CacheCfg {
  static constexpr int kWarps = WARPS, kThreads = 32 * WARPS;
  static constexpr int kRows = 8 * NT;
  static constexpr int kBlock = page_head_bytes(DH, DV);
  static constexpr int kRing = kWarps * kStages * kBlock;
  static constexpr int kOStride = DV + 4;                  // floats; staggers the rows over the banks
  static constexpr int kMerge = kWarps * kRows * (kOStride + 2) * 4;
  static constexpr int kOffBar = (kRing > kMerge ? kRing : kMerge);
  static constexpr int kOffAbort = kOffBar + kWarps * kStages * 8;
  static constexpr int kSmemBytes = kOffAbort + 8;
  // Resident CTAs per SM that the registers are held to (four warps: 128 of a
  // thread for 8 rows, 168 for 16).  One more where key rows of 64 leave
  // registers and many CTAs take turns: 256 sequences of 2048 keys, 32 heads on
  // 8, 62.3 to 59.7 us, 16 rows on 4 heads 51.2 to 45.0; but not for ranges
  // (16 rows 21.4 to 24.0 us: more of them, each shorter).
  static constexpr int kMore = WHOLE && DH == 64 ? 1 : 0;
  static constexpr int kResident =
      WARPS == kDecodeCacheWideWarps ? 1 : (NT == 1 ? kDecodeCacheResident8 : kDecodeCacheResident16) + kMore;
  static_assert(kBlock % 16 == 0 && kOffBar % 8 == 0, "bulk copies and barriers");
  static_assert(kResident * (kSmemBytes + 1024) <= 233472, "shared memory of the resident CTAs");
};

// WHOLE: every CTA takes one whole sequence.
template <int DH, int DV, int NT, int WARPS, bool WHOLE>
__global__ void __launch_bounds__(WARPS * 32, CacheCfg<DH, DV, NT, WARPS, WHOLE>::kResident)
decode_cache_kernel(const __grid_constant__ DecCacheParams p) {
  using C = CacheCfg<DH, DV, NT, WARPS, WHOLE>;
  constexpr int kWarps = WARPS;
  constexpr int GK = DH / kQuantGroup, GV = DV / kQuantGroup;
  extern __shared__ __align__(128) uint8_t smem[];
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffAbort);
  const uint32_t warp = warp_id();
  const uint32_t lane = lane_id();
  const int g = static_cast<int>(lane >> 2), t = static_cast<int>(lane & 3);

  const uint32_t ring = smem_u32(smem) + warp * kStages * C::kBlock;
  const uint8_t* ring_ptr = smem + warp * kStages * C::kBlock;
  const uint32_t bars = smem_u32(smem) + C::kOffBar + warp * kStages * 8;
  if (threadIdx.x == 0) *abort_flag = status_blocks(p.status) ? 2 : 0;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(bars + 8 * s, 1);
    fence_mbar_init();
  }
  Ranges rg{0, 0};
  if (!WHOLE) rg = page_ranges(p, lane);
  __syncthreads();

  // ---- work: range `range` of the pages, of tile (KV head h, row tile) ----
  const int tile = static_cast<int>(blockIdx.x) / p.ranges;
  const int range = static_cast<int>(blockIdx.x) - tile * p.ranges;
  const int h = tile / p.chunks;
  const int r0 = (tile - h * p.chunks) * C::kRows;
  const int R = p.group * p.n_q;
  const int begin = range * rg.per;
  const int end = begin + rg.per < rg.total ? begin + rg.per : rg.total;
  // The sequence that `begin` lies in, and its first page's place.
  int b = 0, seq0 = 0;
  if (WHOLE) {
    b = range;
    if (threadIdx.x == 0 && tile == 0 && p.lengths[b] > p.max_pages * kPageTokens) record_status(p.status, ATTN_ERR_PAGE);
  } else if (begin >= rg.total) {
    b = p.B;                     // nothing left for this CTA
  } else if (begin > 0) {
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      int incl;
      const int n = scan_pages(p, b0, lane, incl);
      const uint32_t past = __ballot_sync(0xffffffffu, seq0 + incl > begin);
      if (past) {
        const int l = __ffs(past) - 1;
        b = b0 + l;
        seq0 += __shfl_sync(0xffffffffu, incl - n, l);
        break;
      }
      seq0 += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  // The merge kernel's view of the same: per, then each sequence's first page.
  if (blockIdx.x == 0 && warp == 0 && !WHOLE) {
    if (lane == 0) p.first_page[0] = rg.per;
    for (int b0 = 0, at = 0; b0 <= p.B; b0 += 32) {
      int incl;
      const int n = scan_pages(p, b0, lane, incl);
      if (b0 + static_cast<int>(lane) <= p.B) p.first_page[1 + b0 + lane] = at + incl - n;
      at += __shfl_sync(0xffffffffu, incl, 31);
    }
  }

  // The stage of this warp's next page, and the parity that its barrier's
  // phase will have (the stages are used in turn, across sequences).
  uint32_t st = 0, parity = 0;
  auto after = [](uint32_t s) { return s + 1 == kStages ? 0u : s + 1; };
  const int b_end = WHOLE ? b + 1 : p.B;
  for (; b < b_end && *abort_flag != 2; ++b) {
    // This lane's chunks of the query rows.
    uint4 qv[NT][GK][2];
    auto load_q = [&] {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = r0 + 8 * nt + g;
        const uint4* q = reinterpret_cast<const uint4*>(p.Q) +
                         ((static_cast<int64_t>(b) * p.Hkv + h) * R + (r < R ? r : 0)) * (DH / 8);
#pragma unroll
        for (int gk = 0; gk < GK; ++gk)
#pragma unroll
          for (int w = 0; w < 2; ++w) qv[nt][gk][w] = r < R ? q[gk * 8 + 2 * t + w] : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    int ids = 0;            // page numbers of a batch of 32 of this warp's pages, one per lane
    if (WHOLE) {            // what is known without the length, requested along with it
      const int at = static_cast<int>(warp + lane * kWarps);
      if (at < p.max_pages) ids = p.table[static_cast<int64_t>(b) * p.max_pages + at];
      load_q();
    }
    int len;
    const int npages = pages_of(p, b, len);
    // This CTA's pages [first, last) of sequence b.  Sequences without pages
    // are the merge kernel's, where there is one.
    const int next0 = seq0 + npages;
    if (!WHOLE) {
      if (seq0 >= end) break;
      if (npages == 0) continue;
    }
    const int first = begin > seq0 ? begin - seq0 : 0;
    const int last = !WHOLE && end < next0 ? end - seq0 : npages;

    // This warp's pages: first + warp, + kWarps, ...
    const int mine = (last - first - static_cast<int>(warp) + kWarps - 1) / kWarps;
    const int n = mine > 0 ? mine : 0;
    const int32_t* table = p.table + static_cast<int64_t>(b) * p.max_pages + first + warp;
    uint32_t bad = 0u;      // bit s: stage s stands for a page outside the pool
    int issued = 0;
    auto issue = [&](uint32_t s) {           // the next page, into stage s
      if ((issued & 31) == 0 && (!WHOLE || issued > 0))
        ids = issued + static_cast<int>(lane) < n ? table[(issued + static_cast<int>(lane)) * kWarps] : 0;
      const int id = __shfl_sync(0xffffffffu, ids, issued & 31);
      const bool in_pool = id >= 0 && id < p.pages;
      bad = in_pool ? bad & ~(1u << s) : bad | (1u << s);
      if (lane == 0) {
        if (in_pool) {
          mbar_arrive_expect_tx(bars + 8 * s, C::kBlock);
          bulk_load(ring + s * C::kBlock, p.pool + (static_cast<int64_t>(id) * p.Hkv + h) * C::kBlock, C::kBlock,
                    bars + 8 * s);
        } else {
          record_status(p.status, ATTN_ERR_PAGE);
          mbar_arrive(bars + 8 * s);
        }
      }
      ++issued;
    };
    if (!WHOLE) load_q();
    for (uint32_t s = st; issued < kStages && issued < n; s = after(s)) issue(s);

    // ---- Q fragments: column g of row group nt is query row r0 + 8 nt + g ----
    // k-step 4 gk + 2 w + e holds the dims 64 gk + 16 t + 8 w + {2e, 2e+4} in
    // its first and {2e+1, 2e+5} in its second register, the nibbles that one
    // mask takes from a word of codes.
    uint32_t qf[NT][4 * GK][2];
    float f[NT][2];        // scale log2(e) 2^(9 - e) of query rows 2t, 2t+1 of the group
    int lim[NT][2];        // keys below lim are visible to them
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t m = 0u;
#pragma unroll
      for (int gk = 0; gk < GK; ++gk)
#pragma unroll
        for (int w = 0; w < 2; ++w) m = bf16_absmax_fold(m, qv[nt][gk][w]);
      uint32_t mb = __float_as_uint(bf16_absmax_value(m));     // (as bits, so that a NaN is the largest)
      mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
      mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
      const float mx = __uint_as_float(mb);
      // 2^14 <= mx 2^e < 2^15 (0 and non-finite rows: e = 0).
      int e = 0;
      if (mx > 0.f && mx < INFINITY) e = 14 - ilogbf(mx);
      e = e > 120 ? 120 : e;
      const float up = exp2_int(e);
#pragma unroll
      for (int gk = 0; gk < GK; ++gk)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          // x, y: dims 0..3, z, w: dims 4..7 of the 16-byte chunk.
          const uint4 u = bf16x8_to_f16x8_scaled(qv[nt][gk][w], up);
          qf[nt][4 * gk + 2 * w][0] = __byte_perm(u.x, u.z, 0x5410);
          qf[nt][4 * gk + 2 * w][1] = __byte_perm(u.x, u.z, 0x7632);
          qf[nt][4 * gk + 2 * w + 1][0] = __byte_perm(u.y, u.w, 0x5410);
          qf[nt][4 * gk + 2 * w + 1][1] = __byte_perm(u.y, u.w, 0x7632);
        }
      // The factors and limits of the rows this lane has in the accumulators.
      // Never 0, which a masked -inf must not meet; NaN for a row of Q with an
      // infinity or a NaN, whose fp16 operands hide it.
      float fac = fmaxf(p.scale_log2 * exp2_int(-e) * 512.0f, 0x1p-126f);
      if (!(mx < INFINITY)) fac = __uint_as_float(0x7FC00000u);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        f[nt][k] = __shfl_sync(0xffffffffu, fac, (2 * t + k) * 4);
        const int row = r0 + 8 * nt + 2 * t + k;
        lim[nt][k] = row < R ? len - p.n_q + 1 + row % p.n_q : 0;
        if (lim[nt][k] <= 0) f[nt][k] = 0x1p-126f;     // (sees no key: not NaN either)
      }
    }

    // O^T before the zero points, [group][dim pair i][(dim, row), (dim, row + 1),
    // 16 (dim + 1, row), 16 (dim + 1, row + 1)], and what they take off.
    float o[NT][GV][4][4], oz[NT][GV][2];
    float shift[NT][2], l_sum[NT][2];      // less the reference that P is relative to; the sum of P
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int k = 0; k < 2; ++k) shift[nt][k] = -kNoKey, l_sum[nt][k] = 0.f;
#pragma unroll
      for (int gv = 0; gv < GV; ++gv)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k < 2) oz[nt][gv][k] = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) o[nt][gv][i][k] = 0.f;
        }
    }
    // 1 / top, and the scale from which on a weight may be too large for fp16
    // (the least of the lane's rows).
    float w_up[NT][GV][2], s_lim[GV];
#pragma unroll
    for (int gv = 0; gv < GV; ++gv) {
      s_lim[gv] = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) w_up[nt][gv][0] = w_up[nt][gv][1] = exp2_int(-kLeastTop);
    }
    // The row of V's codes that this lane addresses in a transposed load: key
    // (lane & 7), of the second eight from lane 16 on, 16 bytes on for odd
    // groups of eight lanes.
    const uint32_t v_addr = ring + off_v_codes(DH) + ((lane & 7) + (lane >> 4) * 8) * (DV / 2) + ((lane >> 3) & 1) * 16;

    auto add_lanes = [](float x) {             // over the 8 lanes of a query row
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      return x + __shfl_xor_sync(0xffffffffu, x, 16);
    };
    int done = 0;
    while (done < n) {
      if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * st, parity, abort_flag, p.wait_limit_ns))) break;
      {
        const uint8_t* blk = ring_ptr + st * C::kBlock;
        const int key0 = (first + static_cast<int>(warp) + done * kWarps) * kPageTokens;
        // ---- S^T of the page's two 16-key blocks ----
        float s[2][NT][4];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          const int ka = 16 * kb + g;
          uint32_t pa[GK], pb[GK];
          lds_words<GK>(blk + off_k_words(DH, DV) + ka * (GK * 4), pa);
          lds_words<GK>(blk + off_k_words(DH, DV) + (ka + 8) * (GK * 4), pb);
#pragma unroll
          for (int gk = 0; gk < GK; ++gk) {
            const uint8_t* kc = blk + off_k_codes() + gk * 32 + t * 8;
            const uint2 wa = lds64(kc + ka * (DH / 2)), wb = lds64(kc + (ka + 8) * (DH / 2));
            // -z 2^-9 of both keys
            const uint32_t za = hfma2_bits(__byte_perm(pa[gk], 0u, 0x4040), kMinusTwo15, 0u);
            const uint32_t zb = hfma2_bits(__byte_perm(pb[gk], 0u, 0x4040), kMinusTwo15, 0u);
            float acc[NT][4];
#pragma unroll
            for (int step = 0; step < 4; ++step) {
              uint32_t xa = step < 2 ? wa.x : wa.y, xb = step < 2 ? wb.x : wb.y;
              if (step & 1) xa >>= 8, xb >>= 8;
              const uint32_t a0 = hfma2_bits(low_nibbles(xa), kTwo15, za), a1 = hfma2_bits(low_nibbles(xb), kTwo15, zb);
              const uint32_t a2 = hfma2_bits(high_nibbles(xa), kTwo11, za), a3 = hfma2_bits(high_nibbles(xb), kTwo11, zb);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint32_t b0 = qf[nt][4 * gk + step][0], b1 = qf[nt][4 * gk + step][1];
                if (step == 0) mma_f16(acc[nt], a0, a1, a2, a3, b0, b1, 0.f, 0.f, 0.f, 0.f);
                else mma_f16(acc[nt], a0, a1, a2, a3, b0, b1);
              }
            }
            const float sa = bf16_hi(pa[gk]), sb = bf16_hi(pb[gk]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float* x = s[kb][nt];
              if (gk == 0) {
                fmul2(x[0], x[1], acc[nt][0], acc[nt][1], sa, sa);
                fmul2(x[2], x[3], acc[nt][2], acc[nt][3], sb, sb);
              } else {
                ffma2(x[0], x[1], acc[nt][0], acc[nt][1], sa, sa, x[0], x[1]);
                ffma2(x[2], x[3], acc[nt][2], acc[nt][3], sb, sb, x[2], x[3]);
              }
            }
          }
        }
        // ---- the values' words of this lane's four keys, and which keys a
        // row does not see ----  (A word serves as the scale as it is: z in the
        // low bits adds at most 15 2^-23 of it, far below the weights' rounding.)
        uint32_t vw[2][2][GV];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
            lds_words<GV>(blk + off_v_words(DH, DV) + (16 * kb + 8 * hf + g) * (GV * 4), vw[kb][hf]);
        const bool missing = (bad >> st) & 1u;     // (none of a missing page's keys is seen)
        if (missing || key0 + kPageTokens > len - p.n_q + 1) {
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int key = missing ? len : key0 + 16 * kb + 8 * hf + g;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                  if (key >= lim[nt][k]) s[kb][nt][2 * hf + k] = -INFINITY;
              // Slots past the sequence may hold anything: their scale and
              // zero point must not meet a zero weight.
              if (key >= len)
#pragma unroll
                for (int gv = 0; gv < GV; ++gv) vw[kb][hf][gv] = 0u;
            }
        }
        // ---- running maximum (lazy) and the weights' scales ----
        bool need = false;
        float mx[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            mx[nt][k] = fmaxf(fmaxf(s[0][nt][k], s[0][nt][2 + k]), fmaxf(s[1][nt][k], s[1][nt][2 + k]));
            need |= fmaf(mx[nt][k], f[nt][k], shift[nt][k]) > static_cast<float>(kLazy);
          }
#pragma unroll
        for (int gv = 0; gv < GV; ++gv) {
          const float smax = fmax3(fmaxf(__uint_as_float(vw[0][0][gv]), __uint_as_float(vw[0][1][gv])),
                                   __uint_as_float(vw[1][0][gv]), __uint_as_float(vw[1][1][gv]));
          need |= smax > s_lim[gv];
        }
        if (__any_sync(0xffffffffu, need)) {
          float least[GV];
#pragma unroll
          for (int gv = 0; gv < GV; ++gv) least[gv] = INFINITY;
          auto max_lanes = [](float x) {         // over the 8 lanes of a query row
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          };
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float m = ceilf(max_lanes(mx[nt][k]) * f[nt][k]);
              float alpha = 1.f;
              if (m + shift[nt][k] > static_cast<float>(kLazy)) {    // (whole octaves: alpha is a power of two)
                alpha = fast_exp2(-shift[nt][k] - m);
                shift[nt][k] = -m;
              }
              l_sum[nt][k] *= alpha;
              float p[2][2];
#pragma unroll
              for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
                  p[kb][hf] = fast_exp2(fmaf(s[kb][nt][2 * hf + k], f[nt][k], shift[nt][k]));
#pragma unroll
              for (int gv = 0; gv < GV; ++gv) {
                float most = 0.f;                // of the page's P s_j
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                  for (int hf = 0; hf < 2; ++hf) most = fmaxf(most, p[kb][hf] * __uint_as_float(vw[kb][hf][gv]));
                const float was = alpha * inverse_power(w_up[nt][gv][k]);
                const uint32_t at_least = max(near_power(was), static_cast<uint32_t>(127 + kLeastTop) << 23);
                const uint32_t now = max(at_least, next_power(max_lanes(most) * exp2_int(-kTopBits)));
                const float top = __uint_as_float(min(now, static_cast<uint32_t>(127 + kMostTop) << 23));
                w_up[nt][gv][k] = inverse_power(top);
                const float back = was * w_up[nt][gv][k];          // at most 1
                least[gv] = fminf(least[gv], top);
                oz[nt][gv][k] *= back;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  o[nt][gv][i][k] *= back;
                  o[nt][gv][i][2 + k] *= back;
                }
              }
            }
#pragma unroll
          for (int gv = 0; gv < GV; ++gv) s_lim[gv] = least[gv] * exp2_int(kTopBits + kSlack);
        }
        // ---- weights and O^T += V^T P^T ----
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          uint32_t bw[NT][GV][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              float p0, p1;
              ffma2(p0, p1, s[kb][nt][2 * hf], s[kb][nt][2 * hf + 1], f[nt][0], f[nt][1], shift[nt][0], shift[nt][1]);
              p0 = fast_exp2(p0);
              p1 = fast_exp2(p1);
              fadd2(l_sum[nt][0], l_sum[nt][1], p0, p1);
#pragma unroll
              for (int gv = 0; gv < GV; ++gv) {
                const float sc = __uint_as_float(vw[kb][hf][gv]);
                float w0, w1;
                fmul2(w0, w1, p0, p1, w_up[nt][gv][0], w_up[nt][gv][1]);
                fmul2(w0, w1, w0, w1, sc, sc);
                const uint32_t w = pack_half2(w0, w1);
                fma_halves(oz[nt][gv][0], oz[nt][gv][1], w, vw[kb][hf][gv]);    // z as fp16 is z 2^-24
                bw[nt][gv][hf] = transpose8x8(w);
              }
            }
          }
#pragma unroll
          for (int gv = 0; gv < GV; ++gv) {
            uint32_t x[4];         // keys 0-7: dims 4g.. of the group's first and second half; keys 8-15
            load_transposed(v_addr + st * C::kBlock + 16 * kb * (DV / 2) + gv * 32, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t xa = x[i >> 1], xb = x[2 + (i >> 1)];
              if (i & 1) xa >>= 8, xb >>= 8;
              const uint32_t a0 = low_nibbles(xa), a1 = high_nibbles(xa), a2 = low_nibbles(xb), a3 = high_nibbles(xb);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][gv][i], a0, a1, a2, a3, bw[nt][gv][0], bw[nt][gv][1]);
            }
          }
        }
      }
      __syncwarp();            // every lane has read the stage
      if (issued < n) issue(st);
      st = after(st);
      parity ^= st == 0 ? 1u : 0u;
      ++done;
      if (done % kZeroPages == 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int gv = 0; gv < GV; ++gv)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float z = add_lanes(oz[nt][gv][k]);
              oz[nt][gv][k] = 0.f;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                o[nt][gv][i][k] -= z;
                o[nt][gv][i][2 + k] = fmaf(-16.f, z, o[nt][gv][i][2 + k]);
              }
            }
      }
    }
    if (*abort_flag) {
      // Every copy already in flight must land before the CTA can exit.
      int no_abort = 0;
      for (; done < issued; ++done) {
        mbar_wait(bars + 8 * st, parity, &no_abort, p.wait_limit_ns);
        st = after(st);
        parity ^= st == 0 ? 1u : 0u;
      }
    }
    if (!WHOLE && next0 >= end) cudaTriggerProgrammaticLaunchCompletion();   // the merge kernel may start (it waits for this grid)
    __syncthreads();

    // ---- merge of the warps (over the ring) ----
    float* oacc = reinterpret_cast<float*>(smem);                              // [warp][row][kOStride]
    float* mst = oacc + kWarps * C::kRows * C::kOStride;                       // [warp][row]
    float* lst = mst + kWarps * C::kRows;
    // o and oz carry 2^-24 / top (the rows of the high nibbles 2^-20 / top).
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float l = add_lanes(l_sum[nt][k]);
        const int row = static_cast<int>(warp) * C::kRows + 8 * nt + 2 * t + k;
        if (g == 0) {
          mst[row] = -shift[nt][k];
          lst[row] = l;
        }
#pragma unroll
        for (int gv = 0; gv < GV; ++gv) {
          float4* dst = reinterpret_cast<float4*>(oacc + row * C::kOStride + 64 * gv + 4 * g);
          const float z = add_lanes(oz[nt][gv][k]);
          const float up = 16777216.0f * inverse_power(w_up[nt][gv][k]);
          auto lo = [&](int i) { return (o[nt][gv][i][k] - z) * up; };
          auto hi = [&](int i) { return fmaf(o[nt][gv][i][2 + k], 0.0625f, -z) * up; };
          dst[0] = make_float4(lo(0), hi(0), lo(1), hi(1));
          dst[8] = make_float4(lo(2), hi(2), lo(3), hi(3));
        }
      }
    __syncthreads();
    if (*abort_flag) break;
    const bool whole = last - first == npages;
    // Parts of split sequences: place 2 range of the tile for the sequence
    // that the range begins in, 2 range + 1 for one that begins inside it.
    const int64_t part = (static_cast<int64_t>(tile) * p.ranges + range) * 2 + (seq0 > begin ? 1 : 0);
    for (int r = static_cast<int>(warp); r < C::kRows && r0 + r < R; r += kWarps) {
      float M = kNoKey;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mst[w * C::kRows + r]);
      float wt[kWarps], L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        wt[w] = fast_exp2(mst[w * C::kRows + r] - M);
        L += lst[w * C::kRows + r] * wt[w];
      }
      const float inv = L > 0.f ? 1.0f / L : (L == 0.f ? 0.f : L);    // (NaN stays NaN)
      const float lse = L == 0.f ? -INFINITY : (M + fast_log2(L)) * kLn2;
      constexpr int kPer = DV / 32;
      float acc[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        acc[k] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          acc[k] = fmaf(wt[w], oacc[(w * C::kRows + r) * C::kOStride + lane * kPer + k], acc[k]);
        acc[k] *= inv;
      }
      if (whole) {
        const int64_t row = (static_cast<int64_t>(b) * p.Hkv + h) * R + r0 + r;
        uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.O) + row * DV + lane * kPer);
#pragma unroll
        for (int k = 0; k < kPer; k += 2) dst[k / 2] = pack_bf16x2(acc[k], acc[k + 1]);
        if (lane == 0) p.LSE[row] = lse;
      } else {
        const int64_t row = part * C::kRows + r;
        float* dst = p.Opart + row * DV + lane * kPer;
#pragma unroll
        for (int k = 0; k < kPer; k += 2) *reinterpret_cast<float2*>(dst + k) = make_float2(acc[k], acc[k + 1]);
        if (lane == 0) p.Lpart[row] = lse;
      }
    }
    seq0 = next0;
    // The ring is free for the next sequence's pages (ordinary accesses
    // before, the copy engine's after).
    fence_proxy_async_smem();
    __syncthreads();
  }
  if (threadIdx.x == 0 && *abort_flag == 1) record_status(p.status, ATTN_ERR_TIMEOUT);
}

// Merge of the parts of a sequence that several ranges share: LSE = M + ln
// sum_s exp(LSE_s - M), O = sum_s exp(LSE_s - LSE) O_s.  ROWS query rows per
// block, each shared by kMergeWarps / ROWS warps, which take every so many parts.
// Launched while the main kernel drains.  Rows of a sequence without pages
// get O = 0, LSE = -inf here.
constexpr int kMergeWarps = 4;
template <int DV, int ROWS>
__global__ void __launch_bounds__(kMergeWarps * 32) decode_cache_merge_kernel(const __grid_constant__ DecCacheParams p) {
  constexpr int kPer = DV / 32, kShare = kMergeWarps / ROWS;
  const int R = p.group * p.n_q;
  const uint32_t lane = lane_id(), warp = warp_id();
  const int r = static_cast<int>(blockIdx.x * ROWS + warp / kShare);    // (b, KV head, row)
  const int who = static_cast<int>(warp) % kShare;
  if (r >= p.B * p.Hkv * R) return;          // (ROWS = 1: never)
  const int bh = r / R, row = r - bh * R;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int chunk = row / p.tile_rows;
  // The row in part 0 of its tile; a part has tile_rows of them.
  const int64_t base_row =
      static_cast<int64_t>(h * p.chunks + chunk) * p.ranges * 2 * p.tile_rows + row - chunk * p.tile_rows;
  cudaGridDependencySynchronize();
  if (status_blocks(p.status)) return;
  const int per = p.first_page[0], seq0 = p.first_page[1 + b], npages = p.first_page[2 + b] - seq0;
  const int i0 = seq0 / per, i1 = (seq0 + npages - 1) / per;
  if (npages > 0 && i0 == i1) return;        // written by the main kernel
  auto part_row = [&](int i) { return base_row + (2 * i + (seq0 > i * per ? 1 : 0)) * p.tile_rows; };
  const int n = npages > 0 ? i1 - i0 + 1 : 0;
  float M = -INFINITY;
  for (int i = static_cast<int>(lane); i < n; i += 32) M = fmaxf(M, p.Lpart[part_row(i0 + i)]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  const float base = M == -INFINITY ? 0.f : M;
  float acc[kPer], sum = 0.f;
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
#pragma unroll 8
  for (int i = who; i < n; i += kShare) {
    const int64_t pr = part_row(i0 + i);
    const float w = fast_exp2((p.Lpart[pr] - base) * kLog2e);
    sum += w;
    const float2* src = reinterpret_cast<const float2*>(p.Opart + pr * DV + lane * kPer);
#pragma unroll
    for (int k = 0; k < kPer; k += 2) {
      const float2 v = src[k / 2];
      acc[k] = fmaf(w, v.x, acc[k]);
      acc[k + 1] = fmaf(w, v.y, acc[k + 1]);
    }
  }
  if constexpr (kShare > 1) {
    __shared__ float acc_s[kShare][DV], sum_s[kShare];
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc_s[who][k * 32 + lane] = acc[k];
    if (lane == 0) sum_s[who] = sum;
    __syncthreads();
    if (who > 0) return;
#pragma unroll
    for (int w = 1; w < kShare; ++w) {
      sum += sum_s[w];
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] += acc_s[w][k * 32 + lane];
    }
  }
  const float inv = sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum);
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.O) + static_cast<int64_t>(r) * DV + lane * kPer);
#pragma unroll
  for (int k = 0; k < kPer; k += 2) dst[k / 2] = pack_bf16x2(acc[k] * inv, acc[k + 1] * inv);
  if (lane == 0) p.LSE[r] = sum == 0.f ? -INFINITY : M + fast_log2(sum) * kLn2;
}

// Up to this many query rows, the merge gives each a block of its own: four
// times the loads in flight for the many parts of few long sequences.
// Measured: 8 long sequences of 32 rows, 4 us against 5; 48 ragged ones of 64
// rows, 6 us against 4 with a warp per row.
constexpr int kMergeBlockRows = 8 * 152;

template <int DH, int DV, int NT, int WARPS, bool WHOLE>
cudaError_t launch_t(const DecCacheParams& p, cudaStream_t stream) {
  using C = CacheCfg<DH, DV, NT, WARPS, WHOLE>;
  auto kern = decode_cache_kernel<DH, DV, NT, WARPS, WHOLE>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(p.Hkv * p.chunks * p.ranges), C::kThreads, C::kSmemBytes, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || WHOLE) return e;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  const int rows = p.B * p.Hkv * p.group * p.n_q;
  if (rows <= kMergeBlockRows) {
    cfg.gridDim = dim3(static_cast<unsigned>(rows));
    return cudaLaunchKernelEx(&cfg, decode_cache_merge_kernel<DV, 1>, p);
  }
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kMergeWarps - 1) / kMergeWarps));
  return cudaLaunchKernelEx(&cfg, decode_cache_merge_kernel<DV, kMergeWarps>, p);
}

template <int DH, int DV>
cudaError_t launch_rows(const DecCacheParams& p, cudaStream_t stream) {
  const bool one = p.tile_rows == 8;
  if (!p.whole_seqs)
    return one ? launch_t<DH, DV, 1, kDecodeCacheWarps, false>(p, stream)
               : launch_t<DH, DV, 2, kDecodeCacheWarps, false>(p, stream);
  if (p.wide)
    return one ? launch_t<DH, DV, 1, kDecodeCacheWideWarps, true>(p, stream)
               : launch_t<DH, DV, 2, kDecodeCacheWideWarps, true>(p, stream);
  return one ? launch_t<DH, DV, 1, kDecodeCacheWarps, true>(p, stream)
             : launch_t<DH, DV, 2, kDecodeCacheWarps, true>(p, stream);
}

}  // namespace

cudaError_t launch_decode_cache(int dh, int dv, const DecCacheParams& p, cudaStream_t stream) {
  if (dh == 128 && dv == 128) return launch_rows<128, 128>(p, stream);
  if (dh == 64 && dv == 64) return launch_rows<64, 64>(p, stream);
  if (dh == 128 && dv == 64) return launch_rows<128, 64>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace esd
