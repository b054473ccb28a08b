// quant_cache.cuh -- the layout of the 4-bit key/value cache.
//
// A pool of pages, each kPageTokens tokens of every KV head:
//   pool [pages][Hkv][page_head_bytes(d_h, d_v)]
// and inside the block of one page and head, in this order:
//   K codes [32][d_h / 2]   V codes [32][d_v / 2]
//   K words [32][d_h / 64]  V words [32][d_v / 64]   (32 bits each)
// Byte i of a row of codes holds element 2i in its low half and 2i + 1 in
// its high half.  The word of a group of 64 elements holds its scale s (bf16)
// in the upper 16 bits and its zero point z (0..15) in the lower 16; an
// element stands for s (code - z).  A block is contiguous and a multiple of
// 16 bytes, so one bulk copy brings it into shared memory.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace esd {

constexpr int kPageTokens = ATTN_CACHE_PAGE_TOKENS;
constexpr int kQuantGroup = 64;    // elements that share a scale and a zero point

__host__ __device__ constexpr int page_head_bytes(int dh, int dv) {
  return kPageTokens * ((dh + dv) / 2 + (dh + dv) / kQuantGroup * 4);
}

// Byte offsets inside a block.
__host__ __device__ constexpr int off_k_codes() { return 0; }
__host__ __device__ constexpr int off_v_codes(int dh) { return kPageTokens * dh / 2; }
__host__ __device__ constexpr int off_k_words(int dh, int dv) { return kPageTokens * (dh + dv) / 2; }
__host__ __device__ constexpr int off_v_words(int dh, int dv) {
  return off_k_words(dh, dv) + kPageTokens * dh / kQuantGroup * 4;
}

}  // namespace esd
