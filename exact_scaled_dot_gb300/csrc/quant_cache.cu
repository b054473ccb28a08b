// quant_cache.cu -- writing tokens into the 4-bit key/value cache and reading
// them back.
//
// A group of 64 elements of a row, lo = min(0, min x) and hi = max(0, max x):
//   s = bf16((hi - lo) / 15),  z = rint(-lo / s),
//   code_i = min(rint(x_i / s) + z, 15),   x_i ~ s (code_i - z),
// (s = 0: every code and z are 0).  0 is always represented exactly.  (s is
// within 2^-8 of (hi - lo) / 15, so z <= 15 and no code is negative.)
//
// The quotients are rounded as exact ones, without dividing.  x and s have 8
// significant bits, so a quotient below 16 either is k + 1/2 exactly or is at
// least 2^-10 away from it; x (1/s) is off by less than 2^-20.  Rounding it to a
// multiple of 2^-11 first (by adding and subtracting 1.5 2^12) therefore puts
// the ties back where they are and moves nothing else across one; adding and
// subtracting 1.5 2^23 then rounds to the integer, ties to even.
//
// Both directions are bound by DRAM (2 bytes per element on one side and
// 0.5625 on the other).  A lane owns 8 elements: one 16-byte access of the
// bf16 row and one 32-bit word of codes; 8 lanes are a group.  A thread keeps
// its place in the token's rows (head, tensor, chunk) and walks over tokens,
// kTokens of them in flight.
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "f16range.cuh"
#include "ptx.cuh"
#include "quant_cache.cuh"

namespace esd {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 4;

constexpr float kToGrid = 6144.0f;          // 1.5 2^12: sums near it are multiples of 2^-11
constexpr float kToInteger = 12582912.0f;   // 1.5 2^23: sums near it are integers

// Larger of two bf16 pairs, element by element.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The lane's eight elements quantised with its group's (eight lanes') range.
__device__ __forceinline__ void quantize8(uint4 v, uint32_t mask, uint32_t& codes, uint32_t& word) {
  // max(0, x) and max(0, -x) over the lane as one pair, then over the group.
  const uint32_t kNeg = 0x80008000u;
  const uint32_t up = max_bf16x2(max_bf16x2(v.x, v.y), max_bf16x2(v.z, v.w));
  const uint32_t dn = max_bf16x2(max_bf16x2(v.x ^ kNeg, v.y ^ kNeg), max_bf16x2(v.z ^ kNeg, v.w ^ kNeg));
  uint32_t m = max_bf16x2(max_bf16x2(__byte_perm(up, dn, 0x5410), __byte_perm(up, dn, 0x7632)), 0u);
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) m = max_bf16x2(m, __shfl_xor_sync(mask, m, off));
  const float hi = bf16_lo(m), neg_lo = bf16_hi(m);
  const uint32_t sb = pack_bf16x2(__fdiv_rn(hi + neg_lo, 15.0f), 0.f) << 16;
  const float s = __uint_as_float(sb);
  float x[8] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y),
                bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w)};
  codes = 0u;
  word = sb;
  if (s < 0x1p-100f) {
    // 1/s may leave fp32's range: divide.  (s = 0: nothing to do.)
    if (s > 0.f) {
      const float z = rintf(__fdiv_rn(neg_lo, s));
#pragma unroll
      for (int k = 0; k < 8; ++k)
        codes |= static_cast<uint32_t>(fminf(rintf(__fdiv_rn(x[k], s)) + z, 15.0f)) << (4 * k);
      word |= static_cast<uint32_t>(z);
    }
    return;
  }
  const float inv = __frcp_rn(s);
  // rint(a / s) + kToInteger: the second sum is exact before its one rounding.
  auto rounded = [inv](float a) { return fmaf(a, inv, kToGrid) + (kToInteger - kToGrid); };
  const float z = rounded(neg_lo) - kToInteger;
  const float back = z - kToInteger;
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = fminf(rounded(x[k]) + back, 15.0f);
  // Four codes in base 16 are an exact fp32 integer.
  const float lo4 = fmaf(fmaf(fmaf(x[3], 16.f, x[2]), 16.f, x[1]), 16.f, x[0]) + 8388608.0f;
  const float hi4 = fmaf(fmaf(fmaf(x[7], 16.f, x[6]), 16.f, x[5]), 16.f, x[4]) + 8388608.0f;
  codes = __byte_perm(__float_as_uint(lo4), __float_as_uint(hi4), 0x5410);
  word |= __float_as_uint(z + 8388608.0f) & 0xFFu;
}

// Blocks of (units, tokens) threads: unit u of a token counts the 8-element
// chunks of K and V of head 0, head 1, ...; blockIdx.y continues the units.
template <bool APPEND, int DH, int DV>
__global__ void __launch_bounds__(kThreads) cache_io_kernel(const __grid_constant__ CacheIoParams p) {
  constexpr int kPer = (DH + DV) / 8;
  const int u = static_cast<int>(blockIdx.y * blockDim.x + threadIdx.x);
  if (u >= p.Hkv * kPer) return;
  // This thread's head, tensor (K or V) and chunk, and where they are in a
  // token's row and, at place 0, in a page.
  const int h = u / kPer;
  const bool val = u - h * kPer >= DH / 8;
  const int c = u - h * kPer - (val ? DH / 8 : 0);
  const int64_t page_stride = static_cast<int64_t>(p.Hkv) * page_head_bytes(DH, DV);
  uint8_t* const head0 = p.pool + static_cast<int64_t>(h) * page_head_bytes(DH, DV);
  uint8_t* const codes0 = head0 + (val ? off_v_codes(DH) : off_k_codes()) + 4 * c;
  uint8_t* const words0 = head0 + (val ? off_v_words(DH, DV) : off_k_words(DH, DV)) + 4 * (c >> 3);
  const int code_row = (val ? DV : DH) / 2, word_row = (val ? DV : DH) / 16;
  const TensorStrides& st = val ? p.sv : p.sk;
  uint4* const rows = static_cast<uint4*>(const_cast<void*>(val ? p.V : p.K)) + h * (st.head / 8) + c;
  const int64_t row = st.row / 8;
  // The eight lanes of a group: their units are consecutive and start at a
  // multiple of 8, as their threads do.
  const uint32_t mask = 0xffu << ((threadIdx.y * blockDim.x + threadIdx.x) & 24u);
  const int tokens = static_cast<int>(p.tokens), step = static_cast<int>(gridDim.x * blockDim.y);
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; t0 < tokens; t0 += kTokens * step) {
    int64_t slot[kTokens];
    uint4 v[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      const int64_t t = t0 + i * static_cast<int64_t>(step);
      slot[i] = t < tokens ? p.slots[t] : -1;
      if (APPEND && t < tokens) v[i] = rows[t * row];
    }
    // Codes and words of the slots; a slot without a token (negative: padding;
    // past the pool: recorded in the status word) has none.
    uint32_t codes[kTokens], word[kTokens];
    int64_t at[kTokens];     // bytes to the slot's page
    int off[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      const bool in_pool = slot[i] < p.pages * kPageTokens;
      if (!in_pool && u == 0) record_status(p.status, ATTN_ERR_PAGE);
      if (!in_pool) slot[i] = -1;
      at[i] = (slot[i] >> 5) * page_stride;
      off[i] = static_cast<int>(slot[i]) & (kPageTokens - 1);
      if (!APPEND) {
        codes[i] = word[i] = 0u;
        if (slot[i] >= 0) {
          codes[i] = *reinterpret_cast<const uint32_t*>(codes0 + at[i] + off[i] * code_row);
          word[i] = *reinterpret_cast<const uint32_t*>(words0 + at[i] + off[i] * word_row);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      const int64_t t = t0 + i * static_cast<int64_t>(step);
      if (APPEND) {
        if (slot[i] < 0) continue;                 // (the same for the group's lanes)
        quantize8(v[i], mask, codes[i], word[i]);
        *reinterpret_cast<uint32_t*>(codes0 + at[i] + off[i] * code_row) = codes[i];
        if ((c & 7) == 0) *reinterpret_cast<uint32_t*>(words0 + at[i] + off[i] * word_row) = word[i];
      } else {
        if (t >= tokens) break;
        const float s = bf16_hi(word[i]);
        // 8388608 + code less 8388608 + z, times s: exact up to the rounding to bf16.
        const float z = __uint_as_float(0x4B000000u | (word[i] & 0xFFu));
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          x[k] = s * (__uint_as_float(0x4B000000u | ((codes[i] >> (4 * k)) & 15u)) - z);
        rows[t * row] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                   pack_bf16x2(x[6], x[7]));
      }
    }
  }
}
static_assert(kPageTokens == 32, "slot >> 5 is the page");

template <bool APPEND, int DH, int DV>
cudaError_t launch_io_t(const CacheIoParams& p, cudaStream_t stream) {
  const int units = p.Hkv * ((DH + DV) / 8);        // a multiple of 16
  const dim3 block(static_cast<unsigned>(std::min(units, kThreads)), static_cast<unsigned>(std::max(1, kThreads / units)));
  // kTokens tokens a thread once there are enough to fill the GPU.
  const int64_t rows = (p.tokens + block.y - 1) / block.y, want = std::max<int64_t>((rows + kTokens - 1) / kTokens, 152 * 4);
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(std::min(rows, want), 152 * 64)),
                  static_cast<unsigned>((units + block.x - 1) / block.x));
  cache_io_kernel<APPEND, DH, DV><<<grid, block, 0, stream>>>(p);
  return cudaGetLastError();
}

template <bool APPEND>
cudaError_t launch_io(const CacheIoParams& p, cudaStream_t stream) {
  if (p.dh == 128 && p.dv == 128) return launch_io_t<APPEND, 128, 128>(p, stream);
  if (p.dh == 64 && p.dv == 64) return launch_io_t<APPEND, 64, 64>(p, stream);
  if (p.dh == 128 && p.dv == 64) return launch_io_t<APPEND, 128, 64>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_cache_append(const CacheIoParams& p, cudaStream_t stream) { return launch_io<true>(p, stream); }

cudaError_t launch_cache_read(const CacheIoParams& p, cudaStream_t stream) { return launch_io<false>(p, stream); }

}  // namespace esd
