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
// several times the traffic of the codes), with the cache as the M side of
// both products and the R = group n_q query rows of a KV head as N = 8 NT
// columns:
//   S^T = K Q^T: A = 16 keys x 16 dims.  A lane's nibbles of one key are its
//     A registers; which dims a lane holds is free as long as Q's fragments
//     agree.  (code - z) is an exact small integer in fp16 and Q is scaled to
//     fp16 by a power of two, exact too (f16range.cuh's argument); the
//     group's scale multiplies the fp32 sums.
//   O^T = V^T P^T: A = 16 dims x 16 keys of exact integers again; the scale
//     goes into the weights, w = P s_j, so each group of 64 dims has a B of its
//     own.  S^T's accumulators, packed to fp16 and transposed 8x8 by
//     movmatrix, are B's registers.
// A nibble becomes fp16 by one logic op against an exponent pattern
// (1024 + c from the low nibbles, 1024 + 16 c from the high ones) and one
// subtraction or fma that removes the offset and z: 1.2 instructions an
// element.
//
// fp16 weights: P <= 2^8 by the lazy running maximum (the reference moves
// only when a score exceeds it by 2^8), times 2^6 s_j 2^-e with 2^e above the
// largest scale seen so far, so w <= 2^14 whatever the values' scale; O is
// rescaled when e grows.  Weights down to 2^-20 of the largest keep 11 bits.
// Sums, maxima and O are fp32.
//
// CTA: 4 warps that share a range of pages of one (sequence, KV head, row
// tile), each with a ring of pages of its own (one bulk copy per page) and
// its own softmax state; no synchronisation until they merge at the end.
// Sequences longer than a range are split over CTAs whose partial results the
// merge kernel joins by their log-sum-exp, as in the decode forward.
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "f16range.cuh"
#include "ptx.cuh"
#include "quant_cache.cuh"

namespace esd {
namespace {

constexpr int kWarps = 4;
constexpr int kStages = 3;
constexpr int kThreads = kWarps * 32;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 8x8 matrix of 16-bit elements spread over the warp (lane 4r + c holds
// columns 2c, 2c+1 of row r), transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

__device__ __forceinline__ uint2 lds64(const uint8_t* p) { return *reinterpret_cast<const uint2*>(p); }
__device__ __forceinline__ uint32_t lds32(const uint8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }

__device__ __forceinline__ uint32_t hadd2_bits(uint32_t a, uint32_t b) {
  const __half2 r = __hadd2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hfma2_bits(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                            *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Bits 0-3 of both halves of x as fp16 c - z: 1024 + c less 1024 + z (nz is
// -(1024 + z) in both halves).  Exact.
__device__ __forceinline__ uint32_t low_nibbles(uint32_t x, uint32_t nz) {
  return hadd2_bits((x & 0x000F000Fu) | 0x64006400u, nz);
}
// Bits 4-7: (1024 + 16 c) / 16 less 64 + z (nz16 is -(64 + z)).  Exact.
__device__ __forceinline__ uint32_t high_nibbles(uint32_t x, uint32_t nz16) {
  return hfma2_bits((x & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, nz16);
}
// -(1024 + z) and -(64 + z) for the zero points z0 (low half) and z1.
__device__ __forceinline__ uint32_t neg_1024(uint32_t z0, uint32_t z1) { return 0xE400E400u | z0 | (z1 << 16); }
__device__ __forceinline__ uint32_t neg_64(uint32_t z0, uint32_t z1) { return 0xD400D400u | (z0 << 4) | (z1 << 20); }

template <int DH, int DV, int NT>
struct CacheCfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kBlock = page_head_bytes(DH, DV);
  static constexpr int kRing = kWarps * kStages * kBlock;
  static constexpr int kOStride = DV + 4;                  // floats; staggers the rows over the banks
  static constexpr int kMerge = kWarps * kRows * (kOStride + 2) * 4;
  static constexpr int kOffBar = (kRing > kMerge ? kRing : kMerge);
  static constexpr int kOffAbort = kOffBar + kWarps * kStages * 8;
  static constexpr int kSmemBytes = kOffAbort + 8;
  static_assert(kBlock % 16 == 0 && kOffBar % 8 == 0, "bulk copies and barriers");
};

template <int DH, int DV, int NT>
__global__ void __launch_bounds__(kThreads)
decode_cache_kernel(const __grid_constant__ DecCacheParams p) {
  using C = CacheCfg<DH, DV, NT>;
  constexpr int GK = DH / kQuantGroup, GV = DV / kQuantGroup;
  extern __shared__ __align__(128) uint8_t smem[];
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffAbort);
  const uint32_t warp = warp_id();
  const uint32_t lane = lane_id();
  const int g = static_cast<int>(lane >> 2), t = static_cast<int>(lane & 3);

  // ---- work item: (sequence, KV head, row tile) and range of pages ----
  const int chunk = static_cast<int>(blockIdx.x) % p.chunks;
  const int bh = static_cast<int>(blockIdx.x) / p.chunks;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int r0 = chunk * C::kRows;
  const int R = p.group * p.n_q;
  const int cap = p.max_pages * kPageTokens;
  int len = p.lengths[b];
  if (len > cap) {
    if (threadIdx.x == 0) record_status(p.status, ATTN_ERR_PAGE);
    len = cap;
  }
  len = len < 0 ? 0 : len;
  const int npages = (len + kPageTokens - 1) / kPageTokens;
  const int first = static_cast<int>(blockIdx.y) * p.split_pages;
  if (first >= npages && blockIdx.y > 0) return;
  const int last = min(first + p.split_pages, npages);

  const uint32_t ring = smem_u32(smem) + warp * kStages * C::kBlock;
  const uint8_t* ring_ptr = smem + warp * kStages * C::kBlock;
  const uint32_t bars = smem_u32(smem) + C::kOffBar + warp * kStages * 8;
  if (threadIdx.x == 0) *abort_flag = status_blocks(p.status) ? 2 : 0;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(bars + 8 * s, 1);
    fence_mbar_init();
  }
  __syncthreads();

  // This warp's pages: first + warp, + kWarps, ...
  const int mine = (last - first - static_cast<int>(warp) + kWarps - 1) / kWarps;
  const int n = mine > 0 && *abort_flag == 0 ? mine : 0;
  const int32_t* table = p.table + static_cast<int64_t>(b) * p.max_pages + first + warp;
  int ids = 0;            // page numbers of a batch of 32 of this warp's pages, one per lane
  uint32_t bad = 0u;      // bit s: stage s stands for a page outside the pool
  auto issue = [&](int it) {
    if ((it & 31) == 0) ids = it + static_cast<int>(lane) < n ? table[(it + static_cast<int>(lane)) * kWarps] : 0;
    const int id = __shfl_sync(0xffffffffu, ids, it & 31);
    const int s = it % kStages;
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
  };
  int issued = 0;
  for (; issued < kStages && issued < n; ++issued) issue(issued);

  // ---- Q fragments: column g of tile nt is query row r0 + 8 nt + g ----
  // k-step 4 gk + 2 w + e holds the dims 64 gk + 16 t + 8 w + {2e, 2e+4} in
  // its first and {2e+1, 2e+5} in its second register, the nibbles that one
  // mask takes from a word of codes.
  uint32_t qf[NT][4 * GK][2];
  float f[NT][2];        // scale log2(e) 2^-e of query rows 2t, 2t+1 of the tile
  int lim[NT][2];        // keys below lim are visible to them
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = r0 + 8 * nt + g;
    const uint4* q = reinterpret_cast<const uint4*>(p.Q) +
                     ((static_cast<int64_t>(b) * p.Hkv + h) * R + (r < R ? r : 0)) * (DH / 8);
    uint4 v[GK][2];
    uint32_t m = 0u;
#pragma unroll
    for (int gk = 0; gk < GK; ++gk)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        v[gk][w] = r < R ? q[gk * 8 + 2 * t + w] : make_uint4(0u, 0u, 0u, 0u);
        m = bf16_absmax_fold(m, v[gk][w]);
      }
    float mx = bf16_absmax_value(m);
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
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
        const uint32_t x = bf16x2_to_f16x2_scaled(v[gk][w].x, up), y = bf16x2_to_f16x2_scaled(v[gk][w].y, up);
        const uint32_t z = bf16x2_to_f16x2_scaled(v[gk][w].z, up), u = bf16x2_to_f16x2_scaled(v[gk][w].w, up);
        qf[nt][4 * gk + 2 * w][0] = __byte_perm(x, z, 0x5410);
        qf[nt][4 * gk + 2 * w][1] = __byte_perm(x, z, 0x7632);
        qf[nt][4 * gk + 2 * w + 1][0] = __byte_perm(y, u, 0x5410);
        qf[nt][4 * gk + 2 * w + 1][1] = __byte_perm(y, u, 0x7632);
      }
    // The factors and limits of the rows this lane has in the accumulators.
    const float fac = p.scale_log2 * exp2_int(-e);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      f[nt][k] = __shfl_sync(0xffffffffu, fac, (2 * t + k) * 4);
      const int row = r0 + 8 * nt + 2 * t + k;
      lim[nt][k] = row < R ? len - p.n_q + 1 + row % p.n_q : 0;
    }
  }

  float o[NT][GV][4][4];     // O^T: [group][dim pair i][(dim, row), (dim, row + 1), (dim + 1, row), (dim + 1, row + 1)]
  float m_ref[NT][2], l_sum[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int k = 0; k < 2; ++k) m_ref[nt][k] = -INFINITY, l_sum[nt][k] = 0.f;
#pragma unroll
    for (int gv = 0; gv < GV; ++gv)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[nt][gv][i][k] = 0.f;
  }
  int e_ref = -100;          // the weights carry 2^(6 - e_ref)
  // Which key of a 16-key block fragment row m (and m + 8) stands for: rows
  // 4q + 2 and 4q + 3 are swapped, so that the four lanes t of one V load
  // read keys of both parities (rows of 64 bytes: both halves of the banks).
  const int key_g = g ^ ((g >> 1) & 1);
  const int key_t0 = (2 * t) ^ (t & 1), key_t1 = (2 * t + 1) ^ (t & 1);

  bool ok = true;
  for (int it = 0; it < n && ok; ++it) {
    const int st = it % kStages;
    ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * st, static_cast<uint32_t>((it / kStages) & 1), abort_flag,
                                           p.wait_limit_ns));
    if (!ok) break;
    if (!((bad >> st) & 1u)) {
      const uint8_t* blk = ring_ptr + st * C::kBlock;
      const int key0 = (first + static_cast<int>(warp) + it * kWarps) * kPageTokens;
      // ---- S^T of the page's two 16-key blocks ----
      float s[2][NT][4];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const int ka = 16 * kb + key_g;
#pragma unroll
        for (int gk = 0; gk < GK; ++gk) {
          const uint8_t* kc = blk + off_k_codes() + gk * 32 + t * 8;
          const uint2 wa = lds64(kc + ka * (DH / 2)), wb = lds64(kc + (ka + 8) * (DH / 2));
          const uint8_t* kw = blk + off_k_words(DH, DV) + gk * 4;
          const uint32_t pa = lds32(kw + ka * (GK * 4)), pb = lds32(kw + (ka + 8) * (GK * 4));
          const uint32_t za = pa & 15u, zb = pb & 15u;
          const uint32_t na = neg_1024(za, za), nb = neg_1024(zb, zb), ha = neg_64(za, za), hb = neg_64(zb, zb);
          float acc[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[nt][k] = 0.f;
#pragma unroll
          for (int step = 0; step < 4; ++step) {
            uint32_t xa = step < 2 ? wa.x : wa.y, xb = step < 2 ? wb.x : wb.y;
            if (step & 1) xa >>= 8, xb >>= 8;
            const uint32_t a0 = low_nibbles(xa, na), a1 = low_nibbles(xb, nb);
            const uint32_t a2 = high_nibbles(xa, ha), a3 = high_nibbles(xb, hb);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(acc[nt], a0, a1, a2, a3, qf[nt][4 * gk + step][0], qf[nt][4 * gk + step][1]);
          }
          const float sa = bf16_hi(pa), sb = bf16_hi(pb);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            s[kb][nt][0] = gk ? fmaf(sa, acc[nt][0], s[kb][nt][0]) : sa * acc[nt][0];
            s[kb][nt][1] = gk ? fmaf(sa, acc[nt][1], s[kb][nt][1]) : sa * acc[nt][1];
            s[kb][nt][2] = gk ? fmaf(sb, acc[nt][2], s[kb][nt][2]) : sb * acc[nt][2];
            s[kb][nt][3] = gk ? fmaf(sb, acc[nt][3], s[kb][nt][3]) : sb * acc[nt][3];
          }
        }
      }
      // ---- the values' scales of this lane's four keys ----
      float sv[2][2][GV];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int gv = 0; gv < GV; ++gv)
            sv[kb][hf][gv] = bf16_hi(lds32(blk + off_v_words(DH, DV) + (16 * kb + 8 * hf + key_g) * (GV * 4) + gv * 4));
      // ---- exp2 domain; keys that a row does not see ----
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[kb][nt][k] *= f[nt][k & 1];
      if (key0 + kPageTokens > len - p.n_q + 1) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int key = key0 + 16 * kb + 8 * hf + key_g;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int k = 0; k < 2; ++k)
                if (key >= lim[nt][k]) s[kb][nt][2 * hf + k] = -INFINITY;
            // Slots past the sequence may hold anything: their scale must
            // not meet a zero weight.
            if (key >= len)
#pragma unroll
              for (int gv = 0; gv < GV; ++gv) sv[kb][hf][gv] = 0.f;
          }
      }
      // ---- running maximum (lazy) and the weights' scale ----
      bool need = false;
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          mx[nt][k] = fmaxf(fmaxf(s[0][nt][k], s[0][nt][2 + k]), fmaxf(s[1][nt][k], s[1][nt][2 + k]));
          need |= mx[nt][k] > m_ref[nt][k] + 8.0f;
        }
      uint32_t smax = 0u;    // bits of the largest scale (non-negative floats order like their bits)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int gv = 0; gv < GV; ++gv) smax = max(smax, __float_as_uint(sv[kb][hf][gv]) & 0x7FFFFFFFu);
      const int e_new = static_cast<int>(smax >> 23) - 126;     // 2^e_new > the largest scale
      need |= e_new > e_ref;
      if (__any_sync(0xffffffffu, need)) {
        const uint32_t all = __reduce_max_sync(0xffffffffu, smax);
        int e = static_cast<int>(all >> 23) - 126;
        e = e > 126 ? 126 : (e < e_ref ? e_ref : e);
        const int de = e_ref - e < -126 ? -126 : e_ref - e;
        const float back = exp2_int(de);
        e_ref = e;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float m = mx[nt][k];
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
            float alpha = 1.f;
            if (m > m_ref[nt][k] + 8.0f || m_ref[nt][k] == -INFINITY) {
              alpha = m_ref[nt][k] == -INFINITY ? 0.f : fast_exp2(m_ref[nt][k] - m);
              m_ref[nt][k] = m;
              l_sum[nt][k] *= alpha;
            }
            alpha *= back;
#pragma unroll
            for (int gv = 0; gv < GV; ++gv)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                o[nt][gv][i][k] *= alpha;
                o[nt][gv][i][2 + k] *= alpha;
              }
          }
      }
      // ---- weights and O^T += V^T P^T ----
      const float up = exp2_int(6 - e_ref);
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        uint32_t bw[NT][GV][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float n0 = m_ref[nt][0] == -INFINITY ? 0.f : m_ref[nt][0];
          const float n1 = m_ref[nt][1] == -INFINITY ? 0.f : m_ref[nt][1];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float p0 = fast_exp2(s[kb][nt][2 * hf] - n0), p1 = fast_exp2(s[kb][nt][2 * hf + 1] - n1);
            l_sum[nt][0] += p0;
            l_sum[nt][1] += p1;
#pragma unroll
            for (int gv = 0; gv < GV; ++gv) {
              const float sc = sv[kb][hf][gv] * up;
              bw[nt][gv][hf] = transpose8x8(pack_f16x2(p0 * sc, p1 * sc));
            }
          }
        }
        const uint8_t* vc = blk + off_v_codes(DH) + 16 * kb * (DV / 2) + g * 4;
        const uint8_t* vw = blk + off_v_words(DH, DV) + 16 * kb * (GV * 4);
#pragma unroll
        for (int gv = 0; gv < GV; ++gv) {
          const uint8_t* c = vc + gv * 32;
          const uint32_t w0 = lds32(c + key_t0 * (DV / 2)), w1 = lds32(c + key_t1 * (DV / 2));
          const uint32_t w2 = lds32(c + (key_t0 + 8) * (DV / 2)), w3 = lds32(c + (key_t1 + 8) * (DV / 2));
          const uint8_t* z = vw + gv * 4;
          const uint32_t z0 = lds32(z + key_t0 * (GV * 4)) & 15u, z1 = lds32(z + key_t1 * (GV * 4)) & 15u;
          const uint32_t z2 = lds32(z + (key_t0 + 8) * (GV * 4)) & 15u, z3 = lds32(z + (key_t1 + 8) * (GV * 4)) & 15u;
          const uint32_t na = neg_1024(z0, z1), nb = neg_1024(z2, z3), ha = neg_64(z0, z1), hb = neg_64(z2, z3);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t xa = __byte_perm(w0, w1, i < 2 ? 0x5410 : 0x7632);
            uint32_t xb = __byte_perm(w2, w3, i < 2 ? 0x5410 : 0x7632);
            if (i & 1) xa >>= 8, xb >>= 8;
            const uint32_t a0 = low_nibbles(xa, na), a2 = low_nibbles(xb, nb);
            const uint32_t a1 = high_nibbles(xa, ha), a3 = high_nibbles(xb, hb);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][gv][i], a0, a1, a2, a3, bw[nt][gv][0], bw[nt][gv][1]);
          }
        }
      }
    }
    __syncwarp();            // every lane has read the stage
    if (issued < n) issue(issued++);
  }
  if (*abort_flag) {
    // Every copy already in flight must land before the CTA can exit.
    int no_abort = 0;
    for (int it = issued > kStages ? issued - kStages : 0; it < issued; ++it)
      mbar_wait(bars + 8 * (it % kStages), static_cast<uint32_t>((it / kStages) & 1), &no_abort, p.wait_limit_ns);
  }
  __syncthreads();

  // ---- merge of the warps (over the ring) ----
  float* oacc = reinterpret_cast<float*>(smem);                              // [warp][row][kOStride]
  float* mst = oacc + kWarps * C::kRows * C::kOStride;                       // [warp][row]
  float* lst = mst + kWarps * C::kRows;
  const float down = exp2_int(e_ref - 6);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float l = l_sum[nt][k];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      const int row = static_cast<int>(warp) * C::kRows + 8 * nt + 2 * t + k;
      if (g == 0) {
        mst[row] = m_ref[nt][k];
        lst[row] = l;
      }
#pragma unroll
      for (int gv = 0; gv < GV; ++gv) {
        float4* dst = reinterpret_cast<float4*>(oacc + row * C::kOStride + 64 * gv + 8 * g);
        dst[0] = make_float4(o[nt][gv][0][k] * down, o[nt][gv][0][2 + k] * down, o[nt][gv][1][k] * down,
                             o[nt][gv][1][2 + k] * down);
        dst[1] = make_float4(o[nt][gv][2][k] * down, o[nt][gv][2][2 + k] * down, o[nt][gv][3][k] * down,
                             o[nt][gv][3][2 + k] * down);
      }
    }
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0 && *abort_flag == 1) record_status(p.status, ATTN_ERR_TIMEOUT);
    return;
  }
  const int64_t rows_total = static_cast<int64_t>(p.B) * p.Hkv * R;
  for (int r = static_cast<int>(warp); r < C::kRows && r0 + r < R; r += kWarps) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mst[w * C::kRows + r]);
    const float base = M == -INFINITY ? 0.f : M;
    float wt[kWarps], L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      wt[w] = fast_exp2(mst[w * C::kRows + r] - base);
      L += lst[w * C::kRows + r] * wt[w];
    }
    const float inv = L > 0.f ? 1.0f / L : (L == 0.f ? 0.f : L);    // (NaN stays NaN)
    const float lse = L == 0.f ? -INFINITY : (M + fast_log2(L)) * kLn2;
    const int64_t row = (static_cast<int64_t>(b) * p.Hkv + h) * R + r0 + r;
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
    if (gridDim.y == 1) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.O) + row * DV + lane * kPer);
#pragma unroll
      for (int k = 0; k < kPer; k += 2) dst[k / 2] = pack_bf16x2(acc[k], acc[k + 1]);
      if (lane == 0) p.LSE[row] = lse;
    } else {
      float* dst = p.Opart + (blockIdx.y * rows_total + row) * DV + lane * kPer;
#pragma unroll
      for (int k = 0; k < kPer; k += 2) *reinterpret_cast<float2*>(dst + k) = make_float2(acc[k], acc[k + 1]);
      if (lane == 0) p.Lpart[blockIdx.y * rows_total + row] = lse;
    }
  }
}

// Merge of the page ranges, one warp per query row: LSE = M + ln sum_s
// exp(LSE_s - M), O = sum_s exp(LSE_s - LSE) O_s over the ranges that the
// sequence's length gives it (the first range always exists).
template <int DV>
__global__ void __launch_bounds__(256) decode_cache_merge_kernel(const __grid_constant__ DecCacheParams p) {
  const int R = p.group * p.n_q;
  const int64_t rows = static_cast<int64_t>(p.B) * p.Hkv * R;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (r >= rows || status_blocks(p.status)) return;
  const uint32_t lane = lane_id();
  const int b = static_cast<int>(r / (static_cast<int64_t>(p.Hkv) * R));
  int len = min(p.lengths[b], p.max_pages * kPageTokens);
  len = len < 0 ? 0 : len;
  const int npages = (len + kPageTokens - 1) / kPageTokens;
  const int splits = max(1, (npages + p.split_pages - 1) / p.split_pages);
  float M = -INFINITY;
  for (int s = 0; s < splits; ++s) M = fmaxf(M, p.Lpart[s * rows + r]);
  const float base = M == -INFINITY ? 0.f : M;
  constexpr int kPer = DV / 32;
  float acc[kPer], sum = 0.f;
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
  for (int s = 0; s < splits; ++s) {
    const float w = fast_exp2((p.Lpart[s * rows + r] - base) * kLog2e);
    sum += w;
    const float2* src = reinterpret_cast<const float2*>(p.Opart + (s * rows + r) * DV + lane * kPer);
#pragma unroll
    for (int k = 0; k < kPer; k += 2) {
      const float2 v = src[k / 2];
      acc[k] = fmaf(w, v.x, acc[k]);
      acc[k + 1] = fmaf(w, v.y, acc[k + 1]);
    }
  }
  const float inv = sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum);
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.O) + r * DV + lane * kPer);
#pragma unroll
  for (int k = 0; k < kPer; k += 2) dst[k / 2] = pack_bf16x2(acc[k] * inv, acc[k + 1] * inv);
  if (lane == 0) p.LSE[r] = sum == 0.f ? -INFINITY : M + fast_log2(sum) * kLn2;
}

template <int DH, int DV, int NT>
cudaError_t launch_t(const DecCacheParams& p, cudaStream_t stream) {
  using C = CacheCfg<DH, DV, NT>;
  auto kern = decode_cache_kernel<DH, DV, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(p.B * p.Hkv * p.chunks), static_cast<unsigned>(p.splits));
  kern<<<grid, kThreads, C::kSmemBytes, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.splits == 1) return e;
  const int64_t rows = static_cast<int64_t>(p.B) * p.Hkv * p.group * p.n_q;
  decode_cache_merge_kernel<DV><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int DH, int DV>
cudaError_t launch_rows(const DecCacheParams& p, cudaStream_t stream) {
  return p.tile_rows == 8 ? launch_t<DH, DV, 1>(p, stream) : launch_t<DH, DV, 2>(p, stream);
}

}  // namespace

cudaError_t launch_decode_cache(int dh, int dv, const DecCacheParams& p, cudaStream_t stream) {
  if (dh == 128 && dv == 128) return launch_rows<128, 128>(p, stream);
  if (dh == 64 && dv == 64) return launch_rows<64, 64>(p, stream);
  if (dh == 128 && dv == 64) return launch_rows<128, 64>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace esd
