// cache_mma.cuh -- what the kernels over the 4-bit cache share: the matrix
// product of warps, codes as fp16 operands, bulk copies of pages, powers of two,
// the pages of all sequences as ranges of CTAs.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "f16range.cuh"
#include "ptx.cuh"
#include "quant_cache.cuh"

namespace esd {
namespace {

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
template <typename Params>
__device__ __forceinline__ int pages_of(const Params& p, int b, int& len) {
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
template <typename Params>
__device__ __forceinline__ Ranges page_ranges(const Params& p, uint32_t lane) {
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
template <typename Params>
__device__ __forceinline__ int scan_pages(const Params& p, int b0, uint32_t lane, int& incl) {
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

// The sequence that page `at` of them all lies in, and its first page's place.
// Called by whole warps.
template <typename Params>
__device__ __forceinline__ int sequence_at(const Params& p, int at, uint32_t lane, int& seq0) {
  int b = 0;
  seq0 = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    int incl;
    const int n = scan_pages(p, b0, lane, incl);
    const uint32_t past = __ballot_sync(0xffffffffu, seq0 + incl > at);
    if (past) {
      const int l = __ffs(past) - 1;
      b = b0 + l;
      seq0 += __shfl_sync(0xffffffffu, incl - n, l);
      break;
    }
    seq0 += __shfl_sync(0xffffffffu, incl, 31);
  }
  return b;
}

}  // namespace
}  // namespace esd
