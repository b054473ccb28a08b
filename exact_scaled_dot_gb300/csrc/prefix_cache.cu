// prefix_cache.cu -- attn_fwd_prefix_cache: attention of a few new queries per
// sequence over a prefix that the whole batch shares and over each sequence's
// own pages of the 4-bit cache, on sm_103a.
//
// The softmax over both is put together from parts: with O_s and LSE_s of the
// keys of part s alone, LSE = ln sum_s exp(LSE_s) and O = sum_s exp(LSE_s -
// LSE) O_s ("Appendix A.10 -- Attention matrices and backpropagation", eqs.
// A.10.1-A.10.3: the same function, its sums taken in another order).  Every
// row sees all of the prefix, so that for a KV head the rows of the whole batch
// are one block of queries and the prefix is read once for many of them.
//
// Three launches: the sequences' own keys (the decode's kernel), the prefix (that
// kernel too or, for many rows, prefix_tile.cu) and the merge.  The first is the one
// with short and with long CTAs, so it goes first: the prefix's CTAs take the places
// that it leaves and wait for its end before they exit, and the merge waits for
// them.  The plan in attn_api.cu has the rules.  Two sequences of up to 40 keys
// behind 500: 7.4 us, three short chains of launch, lengths, pages; the call's 26 to
// 28 us are host time, 9 of them the launches, as many the three tensors.
#include <cstdint>
#include <cuda_runtime.h>

#include "decode_cache_kernel.cuh"

namespace esd {
namespace {

// LSE and O of each query row from its parts: a warp per row, a lane per part for
// the weights, then DV / 32 dims a lane, eight parts in flight.  Launched while the
// kernel before drains.  1024 rows of 20 parts, 10 MB out of the second-level cache:
// 4 to 5 us behind the prefix's kernel.
constexpr int kMergeWarps = 4;
template <int DV>
__global__ void __launch_bounds__(kMergeWarps * 32) prefix_merge_kernel(const __grid_constant__ PrefixMergeParams m) {
  constexpr int kPer = DV / 32, kAhead = 8;
  const DecCacheParams& p = m.own;
  const int R = p.group * p.n_q;
  const uint32_t lane = lane_id();
  const int r = static_cast<int>(blockIdx.x * kMergeWarps + warp_id());    // (b, KV head, row)
  if (r >= p.B * p.Hkv * R) return;
  const int bh = r / R, row = r - bh * R;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  // The row in the prefix's first part, and in its own sequence's.
  const int pre_row = b * R + row, pre_chunk = pre_row / m.tile_rows;
  const int64_t pre = static_cast<int64_t>(h * m.chunks + pre_chunk) * m.splits * m.tile_rows + pre_row -
                      pre_chunk * m.tile_rows;
  const int chunk = row / p.tile_rows;
  const int64_t base_row =
      static_cast<int64_t>(h * p.chunks + chunk) * p.ranges * 2 * p.tile_rows + row - chunk * p.tile_rows;
  cudaGridDependencySynchronize();
  if (status_blocks(p.status)) return;
  const int used = *m.used;
  int per = 1, seq0 = 0, i0 = 0, own = 1;    // (one part, in Oall)
  bool whole = true;
  if (!p.whole_seqs) {
    per = p.first_page[0], seq0 = p.first_page[1 + b];
    const int npages = p.first_page[2 + b] - seq0;
    i0 = seq0 / per;
    own = npages > 0 ? (seq0 + npages - 1) / per - i0 + 1 : 0;
    whole = own == 1;
  }
  const int n = used + own;
  const float* l_own = whole ? p.Lall : p.Lpart;
  const float* o_own = (whole ? p.Oall : p.Opart) + lane * kPer;
  const float* o_pre = m.Opart + lane * kPer;
  // Row of part i of the prefix, or of the sequence.
  auto own_row = [&](int i) -> int64_t {
    const int k = i0 + i;
    return whole ? r : base_row + (2 * k + (seq0 > k * per ? 1 : 0)) * p.tile_rows;
  };
  auto lse_of = [&](int i) {
    return i >= n ? -INFINITY : i < used ? m.Lpart[pre + static_cast<int64_t>(i) * m.tile_rows] : l_own[own_row(i - used)];
  };
  float M = -INFINITY, first = lse_of(static_cast<int>(lane));     // (parts past the 32nd are read twice)
  for (int i = static_cast<int>(lane); i < n; i += 32) M = fmaxf(M, i < 32 ? first : lse_of(i));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  const float base = M == -INFINITY ? 0.f : M;
  float acc[kPer], sum = 0.f;
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
  for (int j0 = 0; j0 < n; j0 += 32) {
    const float w = fast_exp2(((j0 == 0 ? first : lse_of(j0 + static_cast<int>(lane))) - base) * kLog2e);   // (0: none)
    sum += w;
    const int some = n - j0 < 32 ? n - j0 : 32;
    for (int i0_ = 0; i0_ < some; i0_ += kAhead) {
      float v[kAhead][kPer];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = j0 + i0_ + u;
        if (i < n) {
          const float* src =
              i < used ? o_pre + (pre + static_cast<int64_t>(i) * m.tile_rows) * DV : o_own + own_row(i - used) * DV;
          if constexpr (kPer == 4) {
            const float4 x = *reinterpret_cast<const float4*>(src);
            v[u][0] = x.x, v[u][1] = x.y, v[u][2] = x.z, v[u][3] = x.w;
          } else {
            const float2 x = *reinterpret_cast<const float2*>(src);
            v[u][0] = x.x, v[u][1] = x.y;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float wu = __shfl_sync(0xffffffffu, w, (i0_ + u) & 31);
        if (j0 + i0_ + u < n) {
#pragma unroll
          for (int k = 0; k < kPer; ++k) acc[k] = fmaf(wu, v[u][k], acc[k]);
        }
      }
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  const float inv = sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum);
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.O) + static_cast<int64_t>(r) * DV + lane * kPer);
#pragma unroll
  for (int k = 0; k < kPer; k += 2) dst[k / 2] = pack_bf16x2(acc[k] * inv, acc[k + 1] * inv);
  if (lane == 0) p.LSE[r] = sum == 0.f ? -INFINITY : M + fast_log2(sum) * kLn2;
}

template <CacheKind KIND, int DH, int DV, int NT, int WARPS, bool WHOLE>
cudaError_t launch_part(const DecCacheParams& p, cudaStream_t stream) {
  using C = CacheCfg<DH, DV, NT, WARPS, WHOLE>;
  auto kern = decode_cache_kernel<KIND, DH, DV, NT, WARPS, WHOLE>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(kern), C::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  // The prefix starts while the own keys' kernel drains.
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.Hkv * p.chunks * p.ranges));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = KIND == kShared ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int DH, int DV>
cudaError_t launch_own(const DecCacheParams& p, cudaStream_t stream) {
  const bool one = p.tile_rows == 8;
  if (!p.whole_seqs)
    return one ? launch_part<kOwn, DH, DV, 1, kDecodeCacheWarps, false>(p, stream)
               : launch_part<kOwn, DH, DV, 2, kDecodeCacheWarps, false>(p, stream);
  if (p.wide)
    return one ? launch_part<kOwn, DH, DV, 1, kDecodeCacheWideWarps, true>(p, stream)
               : launch_part<kOwn, DH, DV, 2, kDecodeCacheWideWarps, true>(p, stream);
  return one ? launch_part<kOwn, DH, DV, 1, kDecodeCacheWarps, true>(p, stream)
             : launch_part<kOwn, DH, DV, 2, kDecodeCacheWarps, true>(p, stream);
}

template <int DH, int DV>
cudaError_t launch_all(const DecCacheParams& prefix, const PrefixTileParams& tile, const PrefixMergeParams& m,
                       cudaStream_t stream) {
  cudaError_t e = launch_own<DH, DV>(m.own, stream);
  if (e != cudaSuccess) return e;
  e = tile.row_tiles > 0        ? launch_prefix_tile(DH, DV, tile, stream)
      : prefix.tile_rows == 8 ? launch_part<kShared, DH, DV, 1, kDecodeCacheWarps, false>(prefix, stream)
                              : launch_part<kShared, DH, DV, 2, kDecodeCacheWarps, false>(prefix, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  const int rows = m.own.B * m.own.Hkv * m.own.group * m.own.n_q;
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kMergeWarps - 1) / kMergeWarps));
  return cudaLaunchKernelEx(&cfg, prefix_merge_kernel<DV>, m);
}

}  // namespace

cudaError_t launch_prefix_cache(int dh, int dv, const DecCacheParams& prefix, const PrefixTileParams& tile,
                                const PrefixMergeParams& merge, cudaStream_t stream) {
  if (dh == 128 && dv == 128) return launch_all<128, 128>(prefix, tile, merge, stream);
  if (dh == 64 && dv == 64) return launch_all<64, 64>(prefix, tile, merge, stream);
  if (dh == 128 && dv == 64) return launch_all<128, 64>(prefix, tile, merge, stream);
  return cudaErrorInvalidValue;
}

}  // namespace esd
