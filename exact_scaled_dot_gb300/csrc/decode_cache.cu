// decode_cache.cu -- attn_fwd_decode_cache: the kernel over the 4-bit cache
// (decode_cache_kernel.cuh) and the merge of the sequences that several of its
// CTAs share.
#include <cstdint>
#include <cuda_runtime.h>

#include "decode_cache_kernel.cuh"

namespace esd {
namespace {

// Merge of the parts of a sequence that several ranges share: LSE = M + ln
// sum_s exp(LSE_s - M), O = sum_s exp(LSE_s - LSE) O_s.  ROWS query rows per
// block, each shared by kMergeWarps / ROWS warps, which take every so many parts.
// Launched while the main kernel drains.  Rows of a sequence without pages
// get O = 0, LSE = -inf here.
constexpr int kMergeWarps = 4;
template <int DV, int ROWS>
__global__ void __launch_bounds__(kMergeWarps * 32) decode_cache_merge_kernel(const __grid_constant__ DecCacheParams p) {
  constexpr int kPer = DV / 32, kShare = kMergeWarps / ROWS;
  const int R = p.group * p.n_q;
  const uint32_t lane = lane_id(), warp = warp_id();
  const int r = static_cast<int>(blockIdx.x * ROWS + warp / kShare);    // (b, KV head, row)
  const int who = static_cast<int>(warp) % kShare;
  if (r >= p.B * p.Hkv * R) return;          // (ROWS = 1: never)
  const int bh = r / R, row = r - bh * R;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int chunk = row / p.tile_rows;
  // The row in part 0 of its tile; a part has tile_rows of them.
  const int64_t base_row =
      static_cast<int64_t>(h * p.chunks + chunk) * p.ranges * 2 * p.tile_rows + row - chunk * p.tile_rows;
  cudaGridDependencySynchronize();
  if (status_blocks(p.status)) return;
  const int per = p.first_page[0], seq0 = p.first_page[1 + b], npages = p.first_page[2 + b] - seq0;
  const int i0 = seq0 / per, i1 = (seq0 + npages - 1) / per;
  if (npages > 0 && i0 == i1) return;        // written by the main kernel
  auto part_row = [&](int i) { return base_row + (2 * i + (seq0 > i * per ? 1 : 0)) * p.tile_rows; };
  const int n = npages > 0 ? i1 - i0 + 1 : 0;
  float M = -INFINITY;
  for (int i = static_cast<int>(lane); i < n; i += 32) M = fmaxf(M, p.Lpart[part_row(i0 + i)]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  const float base = M == -INFINITY ? 0.f : M;
  float acc[kPer], sum = 0.f;
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
#pragma unroll 8
  for (int i = who; i < n; i += kShare) {
    const int64_t pr = part_row(i0 + i);
    const float w = fast_exp2((p.Lpart[pr] - base) * kLog2e);
    sum += w;
    const float2* src = reinterpret_cast<const float2*>(p.Opart + pr * DV + lane * kPer);
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

// Up to this many query rows, the merge gives each a block of its own: four
// times the loads in flight for the many parts of few long sequences.
// Measured: 8 long sequences of 32 rows, 4 us against 5; 48 ragged ones of 64
// rows, 6 us against 4 with a warp per row.
constexpr int kMergeBlockRows = 8 * 152;

template <int DH, int DV, int NT, int WARPS, bool WHOLE>
cudaError_t launch_t(const DecCacheParams& p, cudaStream_t stream) {
  using C = CacheCfg<DH, DV, NT, WARPS, WHOLE>;
  auto kern = decode_cache_kernel<kDecode, DH, DV, NT, WARPS, WHOLE>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(p.Hkv * p.chunks * p.ranges), C::kThreads, C::kSmemBytes, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || WHOLE) return e;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  const int rows = p.B * p.Hkv * p.group * p.n_q;
  if (rows <= kMergeBlockRows) {
    cfg.gridDim = dim3(static_cast<unsigned>(rows));
    return cudaLaunchKernelEx(&cfg, decode_cache_merge_kernel<DV, 1>, p);
  }
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kMergeWarps - 1) / kMergeWarps));
  return cudaLaunchKernelEx(&cfg, decode_cache_merge_kernel<DV, kMergeWarps>, p);
}

template <int DH, int DV>
cudaError_t launch_rows(const DecCacheParams& p, cudaStream_t stream) {
  const bool one = p.tile_rows == 8;
  if (!p.whole_seqs)
    return one ? launch_t<DH, DV, 1, kDecodeCacheWarps, false>(p, stream)
               : launch_t<DH, DV, 2, kDecodeCacheWarps, false>(p, stream);
  if (p.wide)
    return one ? launch_t<DH, DV, 1, kDecodeCacheWideWarps, true>(p, stream)
               : launch_t<DH, DV, 2, kDecodeCacheWideWarps, true>(p, stream);
  return one ? launch_t<DH, DV, 1, kDecodeCacheWarps, true>(p, stream)
             : launch_t<DH, DV, 2, kDecodeCacheWarps, true>(p, stream);
}

}  // namespace

cudaError_t launch_decode_cache(int dh, int dv, const DecCacheParams& p, cudaStream_t stream) {
  if (dh == 128 && dv == 128) return launch_rows<128, 128>(p, stream);
  if (dh == 64 && dv == 64) return launch_rows<64, 64>(p, stream);
  if (dh == 128 && dv == 64) return launch_rows<128, 64>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace esd
