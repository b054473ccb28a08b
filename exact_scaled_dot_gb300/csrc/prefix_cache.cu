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
#include <cstdint>
#include <cuda_runtime.h>

#include "decode_cache_kernel.cuh"

namespace esd {
namespace {

// LSE and O of each query row from its parts.  ROWS query rows per block, each
// shared by kMergeWarps / ROWS warps, which take every so many parts.
constexpr int kMergeWarps = 4;
template <int DV, int ROWS>
__global__ void __launch_bounds__(kMergeWarps * 32) prefix_merge_kernel(const __grid_constant__ PrefixMergeParams m) {
  constexpr int kPer = DV / 32, kShare = kMergeWarps / ROWS;
  const DecCacheParams& p = m.own;
  const int R = p.group * p.n_q;
  const uint32_t lane = lane_id(), warp = warp_id();
  const int r = static_cast<int>(blockIdx.x * ROWS + warp / kShare);    // (b, KV head, row)
  const int who = static_cast<int>(warp) % kShare;
  if (r >= p.B * p.Hkv * R) return;          // (ROWS = 1: never)
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
  // Row of part i among Opart and Lpart of the prefix or of the sequence, or Oall and Lall.
  auto part_row = [&](int i) -> int64_t {
    if (i < used) return pre + static_cast<int64_t>(i) * m.tile_rows;
    const int k = i0 + i - used;
    return whole ? r : base_row + (2 * k + (seq0 > k * per ? 1 : 0)) * p.tile_rows;
  };
  auto lse_of = [&](int i) { return (i < used ? m.Lpart : whole ? p.Lall : p.Lpart)[part_row(i)]; };
  float M = -INFINITY;
  for (int i = static_cast<int>(lane); i < n; i += 32) M = fmaxf(M, lse_of(i));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  const float base = M == -INFINITY ? 0.f : M;
  float acc[kPer], sum = 0.f;
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
#pragma unroll 4
  for (int i = who; i < n; i += kShare) {
    const float w = fast_exp2((lse_of(i) - base) * kLog2e);
    sum += w;
    const float* part = i < used ? m.Opart : whole ? p.Oall : p.Opart;
    const float2* src = reinterpret_cast<const float2*>(part + part_row(i) * DV + lane * kPer);
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

// Up to this many query rows, the merge gives each a block of its own.
constexpr int kMergeBlockRows = 8 * 152;

template <CacheKind KIND, int DH, int DV, int NT, int WARPS, bool WHOLE>
cudaError_t launch_part(const DecCacheParams& p, cudaStream_t stream) {
  using C = CacheCfg<DH, DV, NT, WARPS, WHOLE>;
  auto kern = decode_cache_kernel<KIND, DH, DV, NT, WARPS, WHOLE>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(p.Hkv * p.chunks * p.ranges), C::kThreads, C::kSmemBytes, stream>>>(p);
  return cudaGetLastError();
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
  cudaError_t e = tile.row_tiles > 0 ? launch_prefix_tile(DH, DV, tile, stream)
                  : prefix.tile_rows == 8 ? launch_part<kShared, DH, DV, 1, kDecodeCacheWarps, false>(prefix, stream)
                                        : launch_part<kShared, DH, DV, 2, kDecodeCacheWarps, false>(prefix, stream);
  if (e != cudaSuccess) return e;
  e = launch_own<DH, DV>(m.own, stream);
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
  if (rows <= kMergeBlockRows) {
    cfg.gridDim = dim3(static_cast<unsigned>(rows));
    return cudaLaunchKernelEx(&cfg, prefix_merge_kernel<DV, 1>, m);
  }
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kMergeWarps - 1) / kMergeWarps));
  return cudaLaunchKernelEx(&cfg, prefix_merge_kernel<DV, kMergeWarps>, m);
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
