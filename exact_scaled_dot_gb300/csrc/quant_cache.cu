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
// Both directions move 2 bytes per element on one side and 0.5625 on the
// other.  A lane owns 8 elements of K's row and 8 of V's: one 16-byte access of
// the bf16 row and one 32-bit word of codes each; 8 lanes are a group.  A
// thread keeps its place in the token's rows (head, chunk) and walks over
// tokens, so that what the two share (slot, page, offsets) is worked out once.
//
// Measured (GB300, 16384 tokens, 8 heads, widths 128): writing and reading
// back 34 us, 76 % of the measured copy rate for their 172 MB.  What bounds both
// is the issue of instructions (0.72 of the schedulers' cycles, the integer
// pipe at 62 %: range, rounding and packing of each element), not DRAM.
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "f16range.cuh"
#include "ptx.cuh"
#include "quant_cache.cuh"

namespace esd {
namespace {

// Threads of a block (16384 tokens, 8 heads, widths 128, writing + reading
// back: 18.7 + 16.1, 19.0 + 16.5, 22.3 + 17.2 us with 128, 256, 512).
constexpr int kThreads = 128;
// Tokens that a thread has in flight once there are enough to fill the GPU
// (the same with 256 threads: 20.4 + 19.0, 19.0 + 16.5, 19.3 + 17.2 and
// 20.6 + 17.0 us with 1, 2, 3 and 4); with fewer, one token a thread.
constexpr int kMostTokens = 2;

constexpr float kToGrid = 6144.0f;          // 1.5 2^12: sums near it are multiples of 2^-11
constexpr float kToInteger = 12582912.0f;   // 1.5 2^23: sums near it are integers

// Pairs of bf16, element by element.
__device__ __forceinline__ __nv_bfloat162 as_pair(uint32_t a) { return *reinterpret_cast<const __nv_bfloat162*>(&a); }
__device__ __forceinline__ uint32_t as_bits(__nv_bfloat162 a) { return *reinterpret_cast<const uint32_t*>(&a); }
__device__ __forceinline__ uint32_t max_pairs(uint32_t a, uint32_t b) { return as_bits(__hmax2(as_pair(a), as_pair(b))); }
__device__ __forceinline__ uint32_t min_pairs(uint32_t a, uint32_t b) { return as_bits(__hmin2(as_pair(a), as_pair(b))); }

// 1/x of a normal x whose reciprocal is normal, within 2^-22 of it.
__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The lane's eight elements quantised with its group's (eight lanes') range.
// Called by whole warps.
__device__ __forceinline__ void quantize8(uint4 v, uint32_t& codes, uint32_t& word) {
  // max(0, x) and max(0, -x) over the lane as one pair, then over the group.
  const uint32_t up = max_pairs(max_pairs(v.x, v.y), max_pairs(v.z, v.w));
  const uint32_t dn = min_pairs(min_pairs(v.x, v.y), min_pairs(v.z, v.w)) ^ 0x80008000u;
  uint32_t m = max_pairs(max_pairs(__byte_perm(up, dn, 0x5410), __byte_perm(up, dn, 0x7632)), 0u);
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) m = max_pairs(m, __shfl_xor_sync(0xffffffffu, m, off));
  const float hi = bf16_lo(m), neg_lo = bf16_hi(m);
  // (hi - lo) / 15 by a product and one correction with the exact remainder,
  // which rounds it correctly (Markstein's theorem) where nothing underflows.
  const float range = hi + neg_lo, q0 = range * (1.0f / 15.0f);
  uint32_t sb = pack_bf16x2(fmaf(fmaf(-15.0f, q0, range), 1.0f / 15.0f, q0), 0.f) << 16;
  float s = __uint_as_float(sb);
  codes = 0u;
  word = 0u;
  if (s < 0x1p-100f) {
    // 1/s may leave fp32's range: divide.  (s = 0: nothing to do.)
    sb = pack_bf16x2(__fdiv_rn(range, 15.0f), 0.f) << 16;
    s = __uint_as_float(sb);
    if (s > 0.f) {
      const float x[8] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y),
                          bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w)};
      const float z = rintf(__fdiv_rn(neg_lo, s));
#pragma unroll
      for (int k = 0; k < 8; ++k)
        codes |= static_cast<uint32_t>(fminf(rintf(__fdiv_rn(x[k], s)) + z, 15.0f)) << (4 * k);
      word = sb | static_cast<uint32_t>(z);
    }
    return;
  }
  const float inv = reciprocal(s);
  // rint(a / s) + kToInteger: the second sum is exact before its one rounding.
  constexpr float kStep = kToInteger - kToGrid;
  const float z = fmaf(neg_lo, inv, kToGrid) + kStep - kToInteger;
  const float back = z - kToInteger;
  // Codes past 15 come from elements above (15 - z) s, which rounded to bf16
  // still is code 15: the elements are cut there, two at a time.
  const float top = (15.0f - z) * s;
  const uint32_t most = pack_bf16x2(top, top);
  v = make_uint4(min_pairs(v.x, most), min_pairs(v.y, most), min_pairs(v.z, most), min_pairs(v.w, most));
  // Pairs (k, k + 4), whose codes go to the same place of the two halves.
  float lo[4] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
  float up4[4] = {bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w)};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    ffma2(lo[k], up4[k], lo[k], up4[k], inv, inv, kToGrid, kToGrid);
    fadd2(lo[k], up4[k], kStep, kStep);
    fadd2(lo[k], up4[k], back, back);
  }
  // Four codes in base 16 are an exact fp32 integer.
#pragma unroll
  for (int k = 2; k >= 0; --k) ffma2(lo[3], up4[3], lo[3], up4[3], 16.f, 16.f, lo[k], up4[k]);
  fadd2(lo[3], up4[3], 8388608.0f, 8388608.0f);
  codes = __byte_perm(__float_as_uint(lo[3]), __float_as_uint(up4[3]), 0x5410);
  word = sb | (__float_as_uint(z + 8388608.0f) & 0xFFu);
}

// Eight elements as bf16: 128 + code less 128 + z, exact, times s, rounded once.
__device__ __forceinline__ uint4 dequantize8(uint32_t codes, uint32_t word) {
  const __nv_bfloat162 z = as_pair(0x43004300u | __byte_perm(word, 0u, 0x4040));
  const __nv_bfloat162 s = as_pair(__byte_perm(word, 0u, 0x3232));
  uint32_t x[4];       // elements (k, k + 4)
#pragma unroll
  for (int k = 0; k < 4; ++k)
    x[k] = as_bits(__hmul2(s, __hsub2(as_pair(((codes >> (4 * k)) & 0x000F000Fu) | 0x43004300u), z)));
  return make_uint4(__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410), __byte_perm(x[0], x[1], 0x7632),
                    __byte_perm(x[2], x[3], 0x7632));
}

// Blocks of (units, tokens) threads: a unit is an 8-element chunk of one head,
// of K's row and (where V's is as wide) of V's; blockIdx.y continues the units.
template <bool APPEND, int DH, int DV, int kTokens>
__global__ void __launch_bounds__(kThreads) cache_io_kernel(const __grid_constant__ CacheIoParams p) {
  constexpr int kPer = DH / 8;
  static_assert(DV <= DH, "V's chunks are among K's");
  const int u = static_cast<int>(blockIdx.y * blockDim.x + threadIdx.x);
  const bool on = u < p.Hkv * kPer;
  const int h = on ? u / kPer : 0;
  const int c = on ? u - h * kPer : 0;
  const bool on_v = on && c < DV / 8;
  // Where the chunk is in a token's rows and, at place 0, in a page (a page is
  // below 2^32 bytes).
  const uint32_t page_stride = static_cast<uint32_t>(p.Hkv) * page_head_bytes(DH, DV);
  uint8_t* const head0 = p.pool + static_cast<int64_t>(h) * page_head_bytes(DH, DV) + 4 * c;
  const int word_of_chunk = 4 * (c >> 3) - 4 * c;
  // Tokens of the thread: t, t + step, ...  The warps go through the loop
  // together (quantize8's sums over lanes), tokens past the end left out.
  const uint32_t tokens = static_cast<uint32_t>(p.tokens), step = gridDim.x * blockDim.y;
  uint32_t t = blockIdx.x * blockDim.y + threadIdx.y;
  const int64_t step_k = p.sk.row / 8 * step, step_v = p.sv.row / 8 * step;
  uint4* row_k = static_cast<uint4*>(const_cast<void*>(p.K)) + h * (p.sk.head / 8) + c + t * (p.sk.row / 8);
  uint4* row_v = static_cast<uint4*>(const_cast<void*>(p.V)) + h * (p.sv.head / 8) + c + t * (p.sv.row / 8);
  for (uint32_t t_block = blockIdx.x * blockDim.y; t_block < tokens; t_block += kTokens * step) {
    int64_t slot[kTokens];
    uint4 v[kTokens][2];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      const bool here = on && t + i * step < tokens;
      slot[i] = here ? p.slots[t + i * step] : -1;
      if (APPEND) {
        v[i][0] = here ? row_k[i * step_k] : make_uint4(0u, 0u, 0u, 0u);
        v[i][1] = here && on_v ? row_v[i * step_v] : make_uint4(0u, 0u, 0u, 0u);
      }
    }
    // Codes and words of the slots, K's and V's; a slot without a token
    // (negative: padding; past the pool: recorded in the status word) has none.
    uint32_t codes[kTokens][2], word[kTokens][2];
    uint8_t* at[kTokens];    // the slot's page
    int off[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      if (slot[i] >= p.pages * kPageTokens) {
        if (u == 0) record_status(p.status, ATTN_ERR_PAGE);
        slot[i] = -1;
      }
      off[i] = static_cast<int>(slot[i]) & (kPageTokens - 1);
      at[i] = head0 + static_cast<uint64_t>(static_cast<uint32_t>(slot[i] >> 5)) * page_stride;
      if (!APPEND) {
        codes[i][0] = word[i][0] = codes[i][1] = word[i][1] = 0u;
        if (slot[i] >= 0) {
          codes[i][0] = *reinterpret_cast<const uint32_t*>(at[i] + off_k_codes() + off[i] * (DH / 2));
          word[i][0] = *reinterpret_cast<const uint32_t*>(at[i] + off_k_words(DH, DV) + word_of_chunk + off[i] * (DH / 16));
          if (on_v) {
            codes[i][1] = *reinterpret_cast<const uint32_t*>(at[i] + off_v_codes(DH) + off[i] * (DV / 2));
            word[i][1] =
                *reinterpret_cast<const uint32_t*>(at[i] + off_v_words(DH, DV) + word_of_chunk + off[i] * (DV / 16));
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      if (APPEND) {
        quantize8(v[i][0], codes[i][0], word[i][0]);
        quantize8(v[i][1], codes[i][1], word[i][1]);
        if (slot[i] >= 0) {
          const bool first = (c & 7) == 0;
          *reinterpret_cast<uint32_t*>(at[i] + off_k_codes() + off[i] * (DH / 2)) = codes[i][0];
          if (first)
            *reinterpret_cast<uint32_t*>(at[i] + off_k_words(DH, DV) + word_of_chunk + off[i] * (DH / 16)) = word[i][0];
          if (on_v) {
            *reinterpret_cast<uint32_t*>(at[i] + off_v_codes(DH) + off[i] * (DV / 2)) = codes[i][1];
            if (first)
              *reinterpret_cast<uint32_t*>(at[i] + off_v_words(DH, DV) + word_of_chunk + off[i] * (DV / 16)) = word[i][1];
          }
        }
      } else if (on && t + i * step < tokens) {
        row_k[i * step_k] = dequantize8(codes[i][0], word[i][0]);
        if (on_v) row_v[i * step_v] = dequantize8(codes[i][1], word[i][1]);
      }
    }
    t += kTokens * step;
    row_k += kTokens * step_k;
    row_v += kTokens * step_v;
  }
}
static_assert(kPageTokens == 32, "slot >> 5 is the page");

constexpr int64_t kFewBlocks = 152 * 4;

template <bool APPEND, int DH, int DV>
cudaError_t launch_io_t(const CacheIoParams& p, cudaStream_t stream) {
  // Blocks of whole warps: several tokens of all units where that fits, else
  // the units rounded up.  Units are a multiple of 8, so the eight lanes of a
  // group are the same token's.
  const int units = p.Hkv * (DH / 8);
  int x = std::min(units, kThreads), y = kThreads / x;
  while (x * y % 32 != 0 && y > 0) --y;
  if (y == 0) {
    x = (x + 31) / 32 * 32;
    y = std::max(1, kThreads / x);
  }
  const dim3 block(static_cast<unsigned>(x), static_cast<unsigned>(y));
  const int64_t rows = (p.tokens + block.y - 1) / block.y;
  const unsigned parts = static_cast<unsigned>((units + block.x - 1) / block.x);
  if (rows * parts <= kFewBlocks) {
    cache_io_kernel<APPEND, DH, DV, 1><<<dim3(static_cast<unsigned>(rows), parts), block, 0, stream>>>(p);
  } else {
    const int64_t x_blocks = std::max<int64_t>((rows + kMostTokens - 1) / kMostTokens, kFewBlocks / parts);
    cache_io_kernel<APPEND, DH, DV, kMostTokens>
        <<<dim3(static_cast<unsigned>(std::min<int64_t>(x_blocks, 152 * 64)), parts), block, 0, stream>>>(p);
  }
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
