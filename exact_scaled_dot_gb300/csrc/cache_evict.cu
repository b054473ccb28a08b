// cache_evict.cu -- attn_cache_evict: every KV head of a sequence that has
// outgrown its budget keeps its first tokens, its newest and those with the most
// attention weight, which move to the front of the sequence's pages.
//
// Of n tokens m = keep stay: the places below `first`, the last `recent` and,
// of those between, the keep - first - recent with the largest weights (equal
// ones: the lowest places).  Softmax does not mind the order of its keys, so a
// token that stays and whose place is below m - recent is left where it is; the
// places there that become free take, in ascending order, the tokens that stay
// from the places behind.  The newest follow in their order.  A steady state
// (a few tokens past the budget) then moves a few tokens and the newest, not
// the whole cache.
//
// The smallest weight that stays is found by its digits, most significant
// first: the weights as integers in their order, a histogram of 11, 11 and 10
// bits of those that agree with the digits so far.  Then each warp counts, in a
// stretch of its own, the tokens that make places free and those that move;
// sums over the warps give every one its rank, without atomics on the lists.
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "f16range.cuh"
#include "ptx.cuh"
#include "quant_cache.cuh"

namespace esd {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kUnroll = 4;

// Weights as integers that order like them: NaN above all, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(w);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  if (w == 0.f) return 0x80000000u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A token of one head in the pool, in pieces: 16 bytes of codes or one 32-bit
// word of a group.
template <int DH, int DV>
struct Token {
  static constexpr int kK = DH / 32, kV = DV / 32, kKw = DH / kQuantGroup, kVw = DV / kQuantGroup;
  static constexpr int kPieces = kK + kV + kKw + kVw;
  // Byte of a piece in the block of a page and head, for the token at `at`.
  __device__ static __forceinline__ int offset(int piece, int at) {
    if (piece < kK) return off_k_codes() + at * (DH / 2) + 16 * piece;
    piece -= kK;
    if (piece < kV) return off_v_codes(DH) + at * (DV / 2) + 16 * piece;
    piece -= kV;
    if (piece < kKw) return off_k_words(DH, DV) + at * (4 * kKw) + 4 * piece;
    return off_v_words(DH, DV) + at * (4 * kVw) + 4 * (piece - kKw);
  }
};

template <int DH, int DV>
__global__ void __launch_bounds__(kThreads) cache_evict_kernel(const __grid_constant__ CacheEvictParams p) {
  using T = Token<DH, DV>;
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t warp_sum[kWarps];
  __shared__ uint32_t found[3];          // a digit, what is still to be taken at it, how many have it
  __shared__ int warp_a[kWarps], warp_b[kWarps];
  const uint32_t warp = warp_id(), lane = lane_id();
  const int tid = static_cast<int>(threadIdx.x);
  const int b = static_cast<int>(blockIdx.x) / p.Hkv, h = static_cast<int>(blockIdx.x) - b * p.Hkv;
  const int cap = p.max_pages * kPageTokens;
  if (status_blocks(p.status)) return;
  int n = p.lengths[b];
  if (n > cap && h == 0 && tid == 0) record_status(p.status, ATTN_ERR_PAGE);
  n = n < 0 ? 0 : (n > cap ? cap : n);
  const int m = n < p.keep ? n : p.keep;
  if (h == 0 && tid == 0) p.new_lengths[b] = m;
  const int64_t bh = static_cast<int64_t>(b) * p.Hkv + h;
  const float* w = p.weights + bh * cap;
  float* nw = p.new_weights + bh * cap;
  int32_t* kept = p.kept ? p.kept + bh * p.keep : nullptr;
  const bool in_place = nw == w;
  if (n <= p.keep) {
    for (int j = tid; j < cap; j += kThreads)
      if (!in_place || j >= n) nw[j] = j < n ? w[j] : 0.f;
    if (kept)
      for (int j = tid; j < p.keep; j += kThreads) kept[j] = j < n ? j : -1;
    return;
  }
  const int c0 = p.first, c1 = n - p.recent;     // the candidates' places
  const int front = m - p.recent;                // places below it keep their token or take one from behind

  // ---- the smallest key that stays, and how many of its equals ----
  uint32_t least = 0xFFFFFFFFu, equals = 0u, had = 0u;
  uint32_t take = static_cast<uint32_t>(p.keep - p.first - p.recent);
  if (take > 0) {
    uint32_t above = 0u;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int low = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0u;
      __syncthreads();
      for (int j0 = c0; j0 < c1; j0 += kThreads * kUnroll) {
        float x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int j = j0 + u * kThreads + tid;
          x[u] = j < c1 ? w[j] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const uint32_t key = order_key(x[u]);
          const bool in = j0 + u * kThreads + tid < c1 && (pass == 0 || key >> (low + bits) == above);
          const uint32_t digit = (key >> low) & ((1u << bits) - 1u);
          // Warps whose keys are all alike (weights that are still 0) add once.
          const uint32_t who = __ballot_sync(0xffffffffu, in);
          if (who == 0u) continue;
          const uint32_t lead = __shfl_sync(0xffffffffu, digit, __ffs(who) - 1);
          if (__all_sync(0xffffffffu, !in || digit == lead)) {
            if (lane == 0) atomicAdd(&hist[lead], static_cast<uint32_t>(__popc(who)));
          } else if (in) {
            atomicAdd(&hist[digit], 1u);
          }
        }
      }
      __syncthreads();
      // From the largest digit down: this thread's bins, and those above them.
      constexpr int kOwn = kBins / kThreads;
      uint32_t mine[kOwn], sum = 0u;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        mine[i] = hist[kBins - 1 - (tid * kOwn + i)];
        sum += mine[i];
      }
      uint32_t incl = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, off);
        if (static_cast<int>(lane) >= off) incl += v;
      }
      if (lane == 31) warp_sum[warp] = incl;
      __syncthreads();
      uint32_t before = incl - sum;
      for (uint32_t k = 0; k < warp; ++k) before += warp_sum[k];
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        if (before < take && take <= before + mine[i]) {
          found[0] = static_cast<uint32_t>(kBins - 1 - (tid * kOwn + i));
          found[1] = take - before;
          found[2] = mine[i];
        }
        before += mine[i];
      }
      __syncthreads();
      above = (above << bits) | found[0];
      take = found[1];
      had = found[2];
    }
    least = above;
    equals = take;
  }

  // ---- each warp's stretch of the candidates: ranks of equals, counts ----
  const int per = ((c1 - c0 + kWarps * 32 - 1) / (kWarps * 32)) * 32;
  const int s0 = c0 + static_cast<int>(warp) * per, s1 = s0 + per < c1 ? s0 + per : c1;
  // Sum over the warps before this one (all warps call it).
  auto before_me = [&](int mine, int* cell) {
    if (lane == 0) cell[warp] = mine;
    __syncthreads();
    int sum = 0;
    for (uint32_t k = 0; k < warp; ++k) sum += cell[k];
    return sum;
  };
  int eq0 = 0;
  const bool some = equals < had;         // not all of the equals stay: the lowest places do
  if (some) {
    int c = 0;
    for (int j = s0 + static_cast<int>(lane); j - static_cast<int>(lane) < s1; j += 32)
      c += __popc(__ballot_sync(0xffffffffu, j < s1 && order_key(w[j]) == least));
    eq0 = before_me(c, warp_a);
    __syncthreads();
  }
  const uint32_t below = (1u << lane) - 1u;
  int eq = eq0;
  // Whether the candidate at j stays; called for 32 of them in order.
  auto stays = [&](int j) {
    const uint32_t key = j < s1 ? order_key(w[j]) : 0u;
    bool yes = j < s1 && key > least;
    if (equals > 0u) {
      const bool is = j < s1 && key == least;
      if (some) {
        const uint32_t all = __ballot_sync(0xffffffffu, is);
        yes |= is && static_cast<uint32_t>(eq + __popc(all & below)) < equals;
        eq += __popc(all);
      } else {
        yes |= is;
      }
    }
    return yes;
  };
  int holes = 0, moves = 0;
  for (int j = s0 + static_cast<int>(lane); j - static_cast<int>(lane) < s1; j += 32) {
    const bool yes = stays(j);
    holes += __popc(__ballot_sync(0xffffffffu, j < s1 && !yes && j < front));
    moves += __popc(__ballot_sync(0xffffffffu, yes && j >= front));
  }
  int hole = before_me(holes, warp_a), move = before_me(moves, warp_b);
  int total = 0;
  for (int k = 0; k < kWarps; ++k) total += warp_b[k];
  int32_t* from = p.lists + bh * 2 * p.most_moves;      // tokens that move, and where to
  int32_t* to = from + p.most_moves;
  eq = eq0;
  for (int j = s0 + static_cast<int>(lane); j - static_cast<int>(lane) < s1; j += 32) {
    const bool yes = stays(j);
    const bool is_hole = j < s1 && !yes && j < front, is_move = yes && j >= front;
    const uint32_t hs = __ballot_sync(0xffffffffu, is_hole), ms = __ballot_sync(0xffffffffu, is_move);
    if (is_hole) to[hole + __popc(hs & below)] = j;
    if (is_move) from[move + __popc(ms & below)] = j;
    hole += __popc(hs);
    move += __popc(ms);
    if (yes && j < front) {
      if (kept) kept[j] = j;
      if (!in_place) nw[j] = w[j];
    }
  }
  for (int j = tid; j < c0; j += kThreads) {
    if (kept) kept[j] = j;
    if (!in_place) nw[j] = w[j];
  }
  __syncthreads();

  // ---- the moves: sources at and behind `front`, places below it ----
  const int32_t* table = p.table + static_cast<int64_t>(b) * p.max_pages;
  auto block_of = [&](int j) -> uint8_t* {       // the block of place j's page and this head, or nullptr
    const int id = table[j / kPageTokens];
    if (id < 0 || id >= p.pages) {
      record_status(p.status, ATTN_ERR_PAGE);
      return nullptr;
    }
    return p.pool + (static_cast<int64_t>(id) * p.Hkv + h) * page_head_bytes(DH, DV);
  };
  auto load_piece = [&](int j, int piece, uint4& v) {
    const uint8_t* src = block_of(j);
    if (!src) return false;
    src += T::offset(piece, j % kPageTokens);
    if (piece < T::kK + T::kV) v = *reinterpret_cast<const uint4*>(src);
    else v.x = *reinterpret_cast<const uint32_t*>(src);
    return true;
  };
  auto store_piece = [&](int j, int piece, uint4 v) {
    uint8_t* dst = block_of(j);
    if (!dst) return;
    dst += T::offset(piece, j % kPageTokens);
    if (piece < T::kK + T::kV) *reinterpret_cast<uint4*>(dst) = v;
    else *reinterpret_cast<uint32_t*>(dst) = v.x;
  };
  for (int i = tid; i < total; i += kThreads) {
    if (kept) kept[to[i]] = from[i];
    nw[to[i]] = w[from[i]];
  }
  const int64_t all_pieces = static_cast<int64_t>(total) * T::kPieces;
  for (int64_t i0 = tid; i0 < all_pieces; i0 += kThreads * kUnroll) {
    uint4 v[kUnroll];
    int at[kUnroll], piece[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t i = i0 + u * kThreads;
      at[u] = -1;
      if (i < all_pieces) {
        const int k = static_cast<int>(i / T::kPieces);
        piece[u] = static_cast<int>(i - static_cast<int64_t>(k) * T::kPieces);
        if (load_piece(from[k], piece[u], v[u])) at[u] = to[k];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (at[u] >= 0) store_piece(at[u], piece[u], v[u]);
  }
  // ---- the newest, in their order: all of a stretch read before it is written ----
  const int shift = n - m;
  __syncthreads();
  for (int i0 = 0; i0 < p.recent; i0 += kThreads) {
    const int i = front + i0 + tid;
    const bool here = i < m;
    const float x = here ? w[i + shift] : 0.f;
    __syncthreads();
    if (here) {
      nw[i] = x;
      if (kept) kept[i] = i + shift;
    }
  }
  const int64_t tail_pieces = static_cast<int64_t>(p.recent) * T::kPieces;
  for (int64_t i0 = 0; i0 < tail_pieces; i0 += kThreads * kUnroll) {
    uint4 v[kUnroll];
    int at[kUnroll], piece[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t i = i0 + u * kThreads + tid;
      at[u] = -1;
      if (i < tail_pieces) {
        const int k = static_cast<int>(i / T::kPieces);
        piece[u] = static_cast<int>(i - static_cast<int64_t>(k) * T::kPieces);
        if (load_piece(front + k + shift, piece[u], v[u])) at[u] = front + k;
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (at[u] >= 0) store_piece(at[u], piece[u], v[u]);
  }
  __syncthreads();
  for (int j = m + tid; j < cap; j += kThreads) nw[j] = 0.f;
}

template <int DH, int DV>
cudaError_t launch_t(const CacheEvictParams& p, cudaStream_t stream) {
  cache_evict_kernel<DH, DV><<<static_cast<unsigned>(p.B * p.Hkv), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_evict(const CacheEvictParams& p, cudaStream_t stream) {
  if (p.dh == 128 && p.dv == 128) return launch_t<128, 128>(p, stream);
  if (p.dh == 64 && p.dv == 64) return launch_t<64, 64>(p, stream);
  if (p.dh == 128 && p.dv == 64) return launch_t<128, 64>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace esd
