// quant_cache.cu -- writing tokens into the 4-bit key/value cache and reading
// them back.
//
// A group of 64 elements of a row, lo = min(0, min x) and hi = max(0, max x):
//   s = bf16((hi - lo) / 15),  z = min(15, rint(-lo / s)),
//   code_i = clamp(rint(x_i / s) + z, 0, 15),   x_i ~ s (code_i - z),
// (s = 0: every code and z are 0).  0 is always represented exactly, and the
// quotients are IEEE divisions, so the codes are the same in any arithmetic
// that rounds them correctly: both operands have 8 significant bits, and such
// a quotient below 16 is either a tie of rint exactly or 2^-17 away from one.
//
// Both directions are bound by DRAM (2 bytes per element on one side and
// 0.5625 on the other).  A lane owns 8 elements: one 16-byte access of the
// bf16 row and one 32-bit word of codes; 8 lanes are a group.
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "f16range.cuh"
#include "ptx.cuh"
#include "quant_cache.cuh"

namespace esd {
namespace {

constexpr int kThreads = 256;

// The lane's eight elements quantised with its group's (eight lanes') range.
__device__ __forceinline__ void quantize8(uint4 v, uint32_t mask, uint32_t& codes, uint32_t& word) {
  float x[8] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y),
                bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w)};
  float lo = 0.f, hi = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    lo = fminf(lo, x[k]);
    hi = fmaxf(hi, x[k]);
  }
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(mask, lo, off));
    hi = fmaxf(hi, __shfl_xor_sync(mask, hi, off));
  }
  const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(hi - lo, 15.0f));
  const float s = __bfloat162float(sb);
  codes = 0u;
  float z = 0.f;
  if (s > 0.f) {
    z = fminf(rintf(__fdiv_rn(-lo, s)), 15.0f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float c = fminf(fmaxf(rintf(__fdiv_rn(x[k], s)) + z, 0.0f), 15.0f);
      codes |= static_cast<uint32_t>(c) << (4 * k);
    }
  }
  word = (static_cast<uint32_t>(__bfloat16_as_ushort(sb)) << 16) | static_cast<uint32_t>(z);
}

// One thread's place: token, head, tensor (0 = K, 1 = V) and 8-element chunk.
// The chunks of a row, K's then V's, run fastest, then the heads.
struct Place {
  int64_t tok;
  int h, c, which;
};
__device__ __forceinline__ Place place_of(const CacheIoParams& p, int64_t u) {
  const int per = (p.dh + p.dv) / 8;
  Place q;
  const int64_t th = u / per;
  int c = static_cast<int>(u - th * per);
  q.which = c >= p.dh / 8 ? 1 : 0;
  q.c = q.which ? c - p.dh / 8 : c;
  q.tok = th / p.Hkv;
  q.h = static_cast<int>(th - q.tok * p.Hkv);
  return q;
}

// The block of the slot's page and head, or nullptr when the slot names no
// token (negative: padding; past the pool: recorded in the status word).
__device__ __forceinline__ uint8_t* slot_block(const CacheIoParams& p, int64_t slot, int h, bool report) {
  if (slot < 0) return nullptr;
  const int64_t page = slot / kPageTokens;
  if (page >= p.pages) {
    if (report) record_status(p.status, ATTN_ERR_PAGE);
    return nullptr;
  }
  return p.pool + (page * p.Hkv + h) * page_head_bytes(p.dh, p.dv);
}

__global__ void __launch_bounds__(kThreads) cache_append_kernel(const __grid_constant__ CacheIoParams p) {
  const int64_t total = p.tokens * p.Hkv * ((p.dh + p.dv) / 8);
  const uint32_t lane = lane_id();
  const uint32_t mask = 0xffu << (lane & 24u);     // the eight lanes of a group
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; u < total;
       u += static_cast<int64_t>(gridDim.x) * kThreads) {
    const Place q = place_of(p, u);
    const int64_t slot = p.slots[q.tok];
    const TensorStrides& st = q.which ? p.sv : p.sk;
    const uint4* src = static_cast<const uint4*>(q.which ? p.V : p.K) + (q.tok * st.row + q.h * st.head) / 8;
    uint8_t* blk = slot_block(p, slot, q.h, q.which == 0 && q.h == 0 && q.c == 0);
    if (!blk) continue;                            // (the same for the group's eight lanes)
    uint32_t codes, word;
    quantize8(src[q.c], mask, codes, word);
    const int off = static_cast<int>(slot % kPageTokens);
    const int d = q.which ? p.dv : p.dh;
    uint8_t* cd = blk + (q.which ? off_v_codes(p.dh) : off_k_codes()) + off * (d / 2);
    reinterpret_cast<uint32_t*>(cd)[q.c] = codes;
    if ((q.c & 7) == 0) {
      uint8_t* wd = blk + (q.which ? off_v_words(p.dh, p.dv) : off_k_words(p.dh, p.dv)) + off * (d / kQuantGroup * 4);
      reinterpret_cast<uint32_t*>(wd)[q.c >> 3] = word;
    }
  }
}

__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheIoParams p) {
  const int64_t total = p.tokens * p.Hkv * ((p.dh + p.dv) / 8);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; u < total;
       u += static_cast<int64_t>(gridDim.x) * kThreads) {
    const Place q = place_of(p, u);
    const int64_t slot = p.slots[q.tok];
    const TensorStrides& st = q.which ? p.sv : p.sk;
    uint4* dst = static_cast<uint4*>(const_cast<void*>(q.which ? p.V : p.K)) + (q.tok * st.row + q.h * st.head) / 8;
    const uint8_t* blk = slot_block(p, slot, q.h, q.which == 0 && q.h == 0 && q.c == 0);
    uint4 out = make_uint4(0u, 0u, 0u, 0u);
    if (blk) {
      const int off = static_cast<int>(slot % kPageTokens);
      const int d = q.which ? p.dv : p.dh;
      const uint8_t* cd = blk + (q.which ? off_v_codes(p.dh) : off_k_codes()) + off * (d / 2);
      const uint8_t* wd =
          blk + (q.which ? off_v_words(p.dh, p.dv) : off_k_words(p.dh, p.dv)) + off * (d / kQuantGroup * 4);
      const uint32_t codes = reinterpret_cast<const uint32_t*>(cd)[q.c];
      const uint32_t word = reinterpret_cast<const uint32_t*>(wd)[q.c >> 3];
      const float s = bf16_hi(word);
      const int z = static_cast<int>(word & 0xFFu);
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = s * static_cast<float>(static_cast<int>((codes >> (4 * k)) & 15u) - z);
      out = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                       pack_bf16x2(x[6], x[7]));
    }
    dst[q.c] = out;
  }
}

unsigned io_blocks(const CacheIoParams& p) {
  int64_t blocks = (p.tokens * p.Hkv * ((p.dh + p.dv) / 8) + kThreads - 1) / kThreads;
  if (blocks > 152 * 64) blocks = 152 * 64;
  return static_cast<unsigned>(blocks);
}

}  // namespace

cudaError_t launch_cache_append(const CacheIoParams& p, cudaStream_t stream) {
  cache_append_kernel<<<io_blocks(p), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheIoParams& p, cudaStream_t stream) {
  cache_read_kernel<<<io_blocks(p), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace esd
