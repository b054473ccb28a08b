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
// bits of those that agree with the digits so far.  Then every thread decides on
// runs of eight tokens, and sums over the threads give the tokens that make
// places free and those that move their ranks, without atomics on the lists.
//
// Work: a CTA per sequence and head, with the weights as integers in its shared
// memory where the page table's places fit.  It moves the tokens too; or, where there
// are few sequences and heads and many tokens may have to move, by the table's places,
// a second kernel with several CTAs for each does: one for the tokens between `front` and m, whose places the
// newest take, and then the newest, the others for those from m on, in whose
// way nothing is.
//
// Measured (GB300, device time).  64 sequences of up to 4128 tokens, 8 heads, widths
// 128, cut to 4096: 20 us for 66 MB, 3.2 TB/s (its floor 9.7).  8 of 16-32 thousand cut
// to 4096: 45 us for 81 MB, 25 and 20 in the two kernels (12).  4 of 513 cut to 512: 9.
// In the first the chain of passes over the keys with a barrier each, the schedulers
// issuing in half of the cycles; in the second 64 CTAs make the lists, and 3000 tokens
// a head are moved 16 bytes here and 8 there (DRAM 42 %, warps that wait for loads).
// A cluster of eight CTAs per head, its histograms added over distributed shared
// memory, was slower than one CTA: a barrier of the cluster for every pass.
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "f16range.cuh"
#include "ptx.cuh"
#include "quant_cache.cuh"

namespace esd {
namespace {

constexpr int kBins = 2048, kPasses = 3;
constexpr int kRun = 8;                   // tokens that a thread decides on at a time
constexpr int kUnroll = 4, kUnrollFirst = 8;
// Threads of a CTA: few where there are many sequences and heads (four CTAs per SM),
// many where there are not.  Weights kept in shared memory, beside histograms of 24
// KB: those of sequences in wider page tables are read from device memory each time,
// short ones too, since the launch knows the table alone.  (Cut from up to 4128 tokens to 4096
// in tables of 129, 192, 193, 512, 1024 pages: 512 heads 19.7, 20.7, 25.1, 27.9, 36.2 us,
// with up to 59 MB of zeros behind the budget; 64 heads 11.1, 17.7, 17.7, 18.3,
// 19.3, from 192 pages on with the second kernel.)  Measured, many against
// few, us (widths 128):
//   4100 tokens cut to 4096: 64 heads 11.0, 13.5; 152 heads 12.0, 13.8; 304 heads 22.0,
//   15.5; 512 heads 40.6, 20.2
//   2048 cut to 1024: 152 heads 13.7, 15.3; 304 heads 25.4, 17.7
//   16384 cut to 1400, past what few threads keep: 152 heads 33.5, 76 and 256 heads 64, 81
// so few from 153 heads on, from 305 on where sequences can be that long.
constexpr int kFewThreads = 256, kManyThreads = 1024;
constexpr int kFewResident = 4, kManyResident = 1;
constexpr int kFewWeights = 6144, kManyWeights = 45056;
constexpr int kManyCtas = 152, kManyLongCtas = 304;
// The second kernel's CTAs per sequence and head and their threads (16 CTAs: 50 us for
// the second case above instead of 45), and the tokens that may move from which on it is
// worth a launch: 16384 cut to 1400, 64 heads, one kernel 23.7 us, two 22.6; 2800 to
// 1400 14.4, 18.6; 16384 to 2400 31.6, 25.5; 4800 to 2400 19.4, 19.8; 16384 to 4096
// 44.7, 30.9.  (With few threads it saves nothing: 304 heads 131, 134 in the last.)
constexpr int kMoveParts = 8, kMoveThreads = 256, kMoveLeast = 2048;

// Weights as integers that order like them: NaN above all, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(w);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  if (w == 0.f) return 0x80000000u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The tokens get(0), get(1) .. of one head to the places put(0), put(1) ..,
// by a CTA, kBatch at a time: first where each is and goes to, then the codes and
// words of K and V, a 16-byte piece or a word a thread and load, so that
// neighbouring tokens are neighbouring addresses.  Everything of a batch is
// requested before any of it is stored; with `between`, after all threads have
// it.  Tokens in or to a page that block_of does not know are left out.
constexpr int kBatch = 256;
struct Moving {
  const uint8_t* src[kBatch];     // the block of the token's page, and of its new one
  uint8_t* dst[kBatch];
  int32_t at[kBatch];             // the places in the pages, the new one times 256
};
template <int DH, int DV, int THREADS, typename Block, typename Get, typename Put>
__device__ __forceinline__ void copy_tokens(Moving& mv, int tid, int count, bool between, Block&& block_of, Get&& get,
                                            Put&& put) {
  static_assert(THREADS >= kBatch, "a thread per token of a batch");
  // K codes, V codes, K words, V words: pieces of a token, and where they are.
  constexpr int kPieces[4] = {DH / 32, DV / 32, DH / kQuantGroup, DV / kQuantGroup};
  constexpr int kAt[4] = {off_k_codes(), off_v_codes(DH), off_k_words(DH, DV), off_v_words(DH, DV)};
  constexpr int kToken[4] = {DH / 2, DV / 2, DH / kQuantGroup * 4, DV / kQuantGroup * 4};
  constexpr int kMost = (kBatch * 4 + THREADS - 1) / THREADS;       // pieces of a thread, of each of the four
  for (int k0 = 0; k0 < count; k0 += kBatch) {
    const int here = count - k0 < kBatch ? count - k0 : kBatch;
    if (tid < here) {
      const int j = get(k0 + tid), to = put(k0 + tid);
      const uint8_t* src = block_of(j);
      mv.src[tid] = src;
      mv.dst[tid] = src ? block_of(to) : nullptr;
      mv.at[tid] = j % kPageTokens | to % kPageTokens << 8;
    }
    __syncthreads();
    uint4 v[2][kMost];
    uint32_t word[2][kMost];
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int u = 0; u < kMost; ++u) {
        const int i = u * THREADS + tid, k = i / kPieces[f], piece = i % kPieces[f];
        if (k < here && mv.dst[k]) {
          const uint8_t* src = mv.src[k] + kAt[f] + piece * (f < 2 ? 16 : 4) + (mv.at[k] & 255) * kToken[f];
          if (f < 2) v[f & 1][u] = *reinterpret_cast<const uint4*>(src);
          else word[f & 1][u] = *reinterpret_cast<const uint32_t*>(src);
        }
      }
    if (between) __syncthreads();
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int u = 0; u < kMost; ++u) {
        const int i = u * THREADS + tid, k = i / kPieces[f], piece = i % kPieces[f];
        if (k < here && mv.dst[k]) {
          uint8_t* dst = mv.dst[k] + kAt[f] + piece * (f < 2 ? 16 : 4) + (mv.at[k] >> 8) * kToken[f];
          if (f < 2) *reinterpret_cast<uint4*>(dst) = v[f & 1][u];
          else *reinterpret_cast<uint32_t*>(dst) = word[f & 1][u];
        }
      }
    __syncthreads();
  }
}

// The block of place j's page and head h in the pool, or nullptr (recorded).
template <int DH, int DV>
__device__ __forceinline__ uint8_t* block_at(const CacheEvictParams& p, const int32_t* table, int h, int j) {
  const int id = table[j / kPageTokens];
  if (id < 0 || id >= p.pages) {
    record_status(p.status, ATTN_ERR_PAGE);
    return nullptr;
  }
  return p.pool + (static_cast<int64_t>(id) * p.Hkv + h) * page_head_bytes(DH, DV);
}

template <int DH, int DV, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == kFewThreads ? kFewResident : kManyResident)
cache_evict_kernel(const __grid_constant__ CacheEvictParams p) {
  constexpr int kThreads = THREADS, kWarps = THREADS / 32;
  extern __shared__ __align__(16) uint32_t smem_words[];
  __shared__ __align__(16) uint32_t hist[kPasses][kBins];
  __shared__ uint32_t found[3];          // a digit, what is still to be taken at it, how many have it
  __shared__ int cells[2][kWarps];       // sums of each warp
  const uint32_t warp = warp_id(), lane = lane_id();
  const int tid = static_cast<int>(threadIdx.x);
  const int bh = static_cast<int>(blockIdx.x);
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int cap = p.max_pages * kPageTokens;
  int n = p.lengths[b];
  const int32_t* table = p.table + static_cast<int64_t>(b) * p.max_pages;
  for (int i = tid; i < kPasses * kBins / 4; i += kThreads) reinterpret_cast<uint4*>(&hist[0][0])[i] = make_uint4(0u, 0u, 0u, 0u);
  if (__syncthreads_or(status_blocks(p.status))) return;
  const bool report = h == 0 && tid == 0;
  if (report && n > cap) record_status(p.status, ATTN_ERR_PAGE);
  n = n < 0 ? 0 : (n > cap ? cap : n);
  const int m = n < p.keep ? n : p.keep;
  if (report) p.new_lengths[b] = m;
  const float* w = p.weights + static_cast<int64_t>(bh) * cap;
  float* nw = p.new_weights + static_cast<int64_t>(bh) * cap;
  int32_t* kept = p.kept ? p.kept + static_cast<int64_t>(bh) * p.keep : nullptr;
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
  const bool held = c1 - c0 <= p.held_weights;
  uint32_t* keys = smem_words;
  // A place that keeps its token (those that do not are written again below).
  auto stay = [&](int j, float x) {
    if (kept) kept[j] = j;
    if (!in_place) nw[j] = x;
  };
  for (int j = tid; j < c0; j += kThreads) stay(j, in_place ? 0.f : w[j]);

  // ---- the smallest key that stays, and how many of its equals ----
  uint32_t least = 0xFFFFFFFFu, equals = 0u, had = 0u;
  uint32_t take = static_cast<uint32_t>(p.keep - p.first - p.recent);
  // (Also with nothing to take: the keys come into shared memory here.)
  for (int j0 = c0; j0 < c1; j0 += kThreads * kUnrollFirst) {
    float x[kUnrollFirst];
#pragma unroll
    for (int u = 0; u < kUnrollFirst; ++u) {
      const int j = j0 + u * kThreads + tid;
      x[u] = j < c1 ? w[j] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kUnrollFirst; ++u) {
      const int j = j0 + u * kThreads + tid;
      if (j < c1) {
        const uint32_t key = order_key(x[u]);
        if (held) keys[j - c0] = key;
        atomicAdd(&hist[0][key >> 21], 1u);
        if (j < front) stay(j, x[u]);
      }
    }
  }
  // (Up to a whole run: 0, which is below every weight's key.)
  if (held && tid < kRun && (c1 - c0) % kRun + tid < kRun && (c1 - c0) % kRun != 0) keys[c1 - c0 + tid] = 0u;
  uint32_t above = 0u;
#pragma unroll 1
  for (int pass = 0; pass < kPasses; ++pass) {
    const int low = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    uint32_t* my_hist = hist[pass];
    if (pass > 0 && held) {
      for (int i = tid * 4; i < c1 - c0; i += kThreads * 4) {
        const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
        const uint32_t four[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (four[u] >> (low + bits) == above) atomicAdd(&my_hist[(four[u] >> low) & ((1u << bits) - 1u)], 1u);
      }
    } else if (pass > 0) {
      for (int j0 = c0; j0 < c1; j0 += kThreads * kUnroll) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int j = j0 + u * kThreads + tid;
          const uint32_t key = j >= c1 ? 0u : order_key(w[j]);
          if (j < c1 && key >> (low + bits) == above) atomicAdd(&my_hist[(key >> low) & ((1u << bits) - 1u)], 1u);
        }
      }
    }
    __syncthreads();
    if (take == 0u) break;
    // From the largest digit down: this thread's bins, and those above them.
    constexpr int kOwn = kBins / kThreads;
    uint32_t mine[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) mine[i] = my_hist[kBins - 1 - tid * kOwn - i];
    uint32_t sum = 0u;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) sum += mine[i];
    uint32_t incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, off);
      if (static_cast<int>(lane) >= off) incl += v;
    }
    if (lane == 31) cells[pass & 1][warp] = static_cast<int>(incl);
    __syncthreads();
    uint32_t before =
        incl - sum + __reduce_add_sync(0xffffffffu, lane < warp ? static_cast<uint32_t>(cells[pass & 1][lane]) : 0u);
    if (before < take && take <= before + sum) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        if (before < take && take <= before + mine[i]) {
          found[0] = static_cast<uint32_t>(kBins - 1 - (tid * kOwn + i));
          found[1] = take - before;
          found[2] = mine[i];
        }
        before += mine[i];
      }
    }
    __syncthreads();
    above = (above << bits) | found[0];
    take = found[1];
    had = found[2];
    least = above;
    equals = take;
    // (found is written again behind the next sync.)
  }

  // ---- who stays: runs of eight tokens a thread, a byte of bits each ----
  uint32_t turn = 0;
  // Sum over the threads before this one, and over all.
  auto before_me = [&](int mine, int& all) {
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, off);
      if (static_cast<int>(lane) >= off) incl += v;
    }
    turn ^= 1u;
    if (lane == 31) cells[turn][warp] = incl;
    __syncthreads();
    const int theirs = lane < kWarps ? cells[turn][lane] : 0;
    all = __reduce_add_sync(0xffffffffu, theirs);
    return incl - mine + __reduce_add_sync(0xffffffffu, lane < warp ? theirs : 0);
  };
  constexpr int kStep = kThreads * kRun;
  const int steps = (c1 - c0 + kStep - 1) / kStep;
  // The bits of a run's tokens that are there, that are above the smallest key, equal to it.
  auto compare = [&](int j, uint32_t& above_it, uint32_t& equal) {
    above_it = equal = 0u;
    if (j >= c1) return;
    uint32_t k[kRun];
    if (held) {
      const uint4 a = *reinterpret_cast<const uint4*>(keys + j - c0), c = *reinterpret_cast<const uint4*>(keys + j - c0 + 4);
      k[0] = a.x, k[1] = a.y, k[2] = a.z, k[3] = a.w, k[4] = c.x, k[5] = c.y, k[6] = c.z, k[7] = c.w;
    } else {
#pragma unroll
      for (int i = 0; i < kRun; ++i) k[i] = j + i < c1 ? order_key(w[j + i]) : 0u;
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      above_it |= k[i] > least ? 1u << i : 0u;
      equal |= k[i] == least ? 1u << i : 0u;
    }
  };
  // The bits of a run's places below `front`.
  auto below_front = [&](int j) { return front - j >= kRun ? 0xFFu : front > j ? (1u << (front - j)) - 1u : 0u; };
  const bool some = equals < had;         // not all of the equals stay: the lowest places do
  int eq = 0;                             // equals before the step
  __syncthreads();                         // (the histograms have been read)
  uint8_t* const bytes = reinterpret_cast<uint8_t*>(&hist[0][0]);
  const bool held_bytes = steps * kThreads <= kPasses * kBins * 4;
  // The run's tokens that stay; with `some`, called by all threads step by step.
  auto decide = [&](int j) {
    uint32_t yes, equal;
    compare(j, yes, equal);
    if (equals > 0u) {
      if (some) {
        int all;
        const int at = eq + before_me(__popc(equal), all);
        eq += all;
        const int left = static_cast<int>(equals) - at;
        while (__popc(equal) > (left > 0 ? left : 0)) equal &= ~(0x80000000u >> __clz(equal));
      }
      yes |= equal;
    }
    return yes;
  };
  int moves = 0;
  for (int i = 0; i < steps; ++i) {
    const int j = c0 + i * kStep + tid * kRun;
    const uint32_t yes = decide(j);
    if (held_bytes) bytes[i * kThreads + tid] = static_cast<uint8_t>(yes);
    const uint32_t low = below_front(j);
    moves += __popc(yes & ~low);
  }
  int hole = 0, move = 0, total;            // before the step
  before_me(moves, total);
  // Tokens that move, and where to: in shared memory where they are few.
  int32_t* from = p.lists ? p.lists + static_cast<int64_t>(bh) * 2 * p.most_moves
                          : reinterpret_cast<int32_t*>(smem_words) + p.held_weights;
  int32_t* to = from + p.most_moves;
  eq = 0;
  for (int i = 0; i < steps; ++i) {
    const int j = c0 + i * kStep + tid * kRun;
    const uint32_t yes = held_bytes ? bytes[i * kThreads + tid] : decide(j);
    const uint32_t there = c1 - j >= kRun ? 0xFFu : c1 > j ? (1u << (c1 - j)) - 1u : 0u, low = below_front(j);
    uint32_t hs = ~yes & there & low, ms = yes & ~low;
    int all;
    const int at = before_me(__popc(hs) | __popc(ms) << 16, all);             // (8192 at most: both in a word)
    int at_hole = hole + (at & 0xFFFF), at_move = move + (at >> 16);
    while (hs) {
      to[at_hole++] = j + __ffs(hs) - 1;
      hs &= hs - 1u;
    }
    while (ms) {
      from[at_move++] = j + __ffs(ms) - 1;
      ms &= ms - 1u;
    }
    hole += all & 0xFFFF;
    move += all >> 16;
  }
  __syncthreads();

  // ---- the moves: sources at and behind `front`, places below it ----
  auto block_of = [&](int j) { return block_at<DH, DV>(p, table, h, j); };
  static_assert(sizeof(Moving) <= sizeof(hist), "over the histograms");
  Moving& mv = *reinterpret_cast<Moving*>(&hist[0][0]);
  for (int i = tid; i < total; i += kThreads) {
    const int j = from[i], to_j = to[i];
    const float x = w[j];
    if (kept) kept[to_j] = j;
    nw[to_j] = x;
  }
  if (p.counts) {
    if (tid == 0) p.counts[bh] = total;
  } else {
    copy_tokens<DH, DV, kThreads>(mv, tid, total, false, block_of, [&](int k) { return from[k]; }, [&](int k) { return to[k]; });
  }
  // ---- the newest, in their order: all of a stretch read before it is written ----
  const int shift = n - m;
  __syncthreads();
  for (int i0 = 0; i0 < p.recent; i0 += kThreads) {
    const int j = front + i0 + tid;
    const float x = j < m ? w[j + shift] : 0.f;
    if (in_place) __syncthreads();
    if (j < m) {
      if (kept) kept[j] = j + shift;
      nw[j] = x;
    }
  }
  if (!p.counts)
    copy_tokens<DH, DV, kThreads>(mv, tid, p.recent, true, block_of, [&](int k) { return front + shift + k; },
                                  [&](int k) { return front + k; });
  __syncthreads();                         // (in place: the newest tokens' weights have been read)
  for (int j = m + tid; j < cap; j += kThreads) nw[j] = 0.f;
}

// The second kernel: the tokens of the lists, and the newest.
template <int DH, int DV>
__global__ void __launch_bounds__(kMoveThreads) cache_move_kernel(const __grid_constant__ CacheEvictParams p) {
  const int tid = static_cast<int>(threadIdx.x);
  const int bh = static_cast<int>(blockIdx.x) / kMoveParts, part = static_cast<int>(blockIdx.x) % kMoveParts;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int cap = p.max_pages * kPageTokens;
  int n = p.lengths[b];
  n = n < 0 ? 0 : (n > cap ? cap : n);
  cudaGridDependencySynchronize();
  if (n <= p.keep) return;
  const int m = p.keep, front = m - p.recent, shift = n - m;
  const int32_t* table = p.table + static_cast<int64_t>(b) * p.max_pages;
  const int32_t* from = p.lists + static_cast<int64_t>(bh) * 2 * p.most_moves;
  const int32_t* to = from + p.most_moves;
  __shared__ Moving mv;
  auto block_of = [&](int j) { return block_at<DH, DV>(p, table, h, j); };
  if (__syncthreads_or(status_blocks(p.status))) return;
  const int total = p.counts[bh];
  // The list ascends: its first `near` tokens come from places below m, where the
  // newest go (at most `recent`; a search by halves would wait for every step's load).
  __shared__ int near_s;
  if (tid == 0) near_s = 0;
  __syncthreads();
  int mine = 0;
  for (int i = tid; i < total && i < p.recent; i += kMoveThreads) mine += from[i] < m;
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane_id() == 0 && mine > 0) atomicAdd(&near_s, mine);
  __syncthreads();
  const int near = near_s;
  if (part == 0) {
    copy_tokens<DH, DV, kMoveThreads>(mv, tid, near, false, block_of, [&](int k) { return from[k]; },
                                      [&](int k) { return to[k]; });
    copy_tokens<DH, DV, kMoveThreads>(mv, tid, p.recent, true, block_of, [&](int k) { return front + shift + k; },
                                      [&](int k) { return front + k; });
  } else {
    const int far = total - near, share = (far + kMoveParts - 2) / (kMoveParts - 1);
    const int k0 = near + (part - 1) * share, k1 = k0 + share < total ? k0 + share : total;
    copy_tokens<DH, DV, kMoveThreads>(mv, tid, k1 - k0, false, block_of, [&](int k) { return from[k0 + k]; },
                                      [&](int k) { return to[k0 + k]; });
  }
}

template <int DH, int DV, int THREADS>
cudaError_t launch_t(CacheEvictParams p, cudaStream_t stream) {
  const int most = THREADS == kFewThreads ? kFewWeights : kManyWeights;
  const int64_t cap = static_cast<int64_t>(p.max_pages) * kPageTokens;
  p.held_weights = cap <= most ? static_cast<int32_t>(cap) : 0;
  const int bytes = (p.held_weights + (p.lists ? 0 : 2 * p.most_moves)) * 4;
  auto kern = cache_evict_kernel<DH, DV, THREADS>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(kern), (most + 2 * kEvictFewMoves) * 4, done);
  if (e != cudaSuccess) return e;
  const bool two = THREADS == kManyThreads && p.most_moves >= kMoveLeast;
  if (!two) p.counts = nullptr;
  kern<<<static_cast<unsigned>(p.B * p.Hkv), THREADS, bytes, stream>>>(p);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess || !two) return err;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B * p.Hkv * kMoveParts));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_move_kernel<DH, DV>, p);
}

template <int DH, int DV>
cudaError_t launch_heads(const CacheEvictParams& p, cudaStream_t stream) {
  const int64_t heads = static_cast<int64_t>(p.B) * p.Hkv, cap = static_cast<int64_t>(p.max_pages) * kPageTokens;
  return heads <= (cap <= kFewWeights ? kManyCtas : kManyLongCtas) ? launch_t<DH, DV, kManyThreads>(p, stream)
                                                                   : launch_t<DH, DV, kFewThreads>(p, stream);
}

}  // namespace

cudaError_t launch_cache_evict(const CacheEvictParams& p, cudaStream_t stream) {
  if (p.dh == 128 && p.dv == 128) return launch_heads<128, 128>(p, stream);
  if (p.dh == 64 && p.dv == 64) return launch_heads<64, 64>(p, stream);
  if (p.dh == 128 && p.dv == 64) return launch_heads<128, 64>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace esd
