// qk_norm.cu -- query and key rows ahead of attention: RMS norm over the head
// width and the rotary position embedding in one pass, its gradients, and the
// rotation alone over several position axes.
//
// A row x of width d (one head of one token), with weights g [d]:
//   r = 1 / sqrt(mean_i x_i^2 + eps),  n = r x,  u = n o g,
//   y_2k   = u_2k cos a_k - u_2k+1 sin a_k
//   y_2k+1 = u_2k sin a_k + u_2k+1 cos a_k,      a_k = pos[axis(k)] w_k
// (blocks beyond the sections have a_k = 0).  With the upstream dy and
// e = R^T dy (dy turned back), t = e o g:
//   dg = sum over rows of e o n
//   dx = r (t - n mean_i(t_i n_i)),
// since d r / d x_i = -r^3 x_i / d.
//
// All three kernels move each row once: 4 bytes per element forward (bf16 in
// and out), 6 backward (x and dy in, dx out), and are bound by DRAM.  A row's
// chunk of 8 elements (one 16-byte access, four blocks) belongs to one lane;
// 16 lanes (8 up to width 64) hold a row and sum over it with shuffles.  A
// lane keeps its chunk for a group of heads of one token, so the token's four
// angles are formed once per group, and every row of the group is requested
// before the first is worked on.
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "ptx.cuh"
#include "rotary.cuh"

namespace esd {
namespace {

constexpr int kThreads = 256;
constexpr int kFwdHeads = 8;    // heads per work item, forward
constexpr int kBwdHeads = 4;    // backward: two rows per head in flight

// The lanes that hold one row.
template <int LANES>
__device__ __forceinline__ uint32_t row_mask(uint32_t lane) {
  return (LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1u)) << (lane & ~(LANES - 1u));
}

template <int LANES>
__device__ __forceinline__ float row_sum(float v, uint32_t mask) {
#pragma unroll
  for (int off = LANES / 2; off > 0; off >>= 1) v += __shfl_xor_sync(mask, v, off);
  return v;
}

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
  x[0] = bf16_lo(v.x), x[1] = bf16_hi(v.x), x[2] = bf16_lo(v.y), x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z), x[5] = bf16_hi(v.z), x[6] = bf16_lo(v.w), x[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// A lane's four blocks: frequencies and axes, fixed for the whole kernel.
struct LaneBlocks {
  float wh[4], wl[4];
  int axis[4];
};
__device__ __forceinline__ LaneBlocks lane_blocks(const QkParams& p, int c) {
  LaneBlocks b;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    b.wh[q] = p.w_hi[4 * c + q];
    b.wl[q] = p.w_lo[4 * c + q];
    b.axis[q] = p.axis[4 * c + q];
  }
  return b;
}

// (cos, sin) of the four blocks at token `tok`: t0 of blocks 0, 1 and t1 of
// blocks 2, 3.  Same angles as the single-axis rotation.
__device__ __forceinline__ void block_angles(const QkParams& p, const LaneBlocks& b, int64_t tok, float4& t0,
                                             float4& t1) {
  if (p.axes == 0) {
    t0 = t1 = make_float4(1.f, 0.f, 1.f, 0.f);
    return;
  }
  int32_t pos[kMaxAxes];
#pragma unroll
  for (int a = 0; a < kMaxAxes; ++a) pos[a] = a < p.axes ? p.pos[a * p.tokens + tok] : 0;
  float c[4], s[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int32_t at = b.axis[q] == 0 ? pos[0] : (b.axis[q] == 1 ? pos[1] : pos[2]);
    rope_cos_sin(reduced_angle(at, b.wh[q], b.wl[q]), c[q], s[q]);
  }
  t0 = make_float4(c[0], s[0], c[1], s[1]);
  t1 = make_float4(c[2], s[2], c[3], s[3]);
}

// Eight fp32 elements turned (s negated by the caller to turn back).
__device__ __forceinline__ void turn8(float (&x)[8], float4 t0, float4 t1) {
  float y0, y1;
  rot_block(x[0], x[1], t0.x, t0.y, y0, y1), x[0] = y0, x[1] = y1;
  rot_block(x[2], x[3], t0.z, t0.w, y0, y1), x[2] = y0, x[3] = y1;
  rot_block(x[4], x[5], t1.x, t1.y, y0, y1), x[4] = y0, x[5] = y1;
  rot_block(x[6], x[7], t1.z, t1.w, y0, y1), x[6] = y0, x[7] = y1;
}

// Weights of a lane's chunk (ones without a weight vector).
__device__ __forceinline__ void load_weights(const void* g, int c, float (&w)[8]) {
  if (g) {
    unpack8(static_cast<const uint4*>(g)[c], w);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = 1.f;
  }
}

// Forward.  Work item: a group of up to kFwdHeads heads of one token; the
// items of the queries come first, then those of the keys.
template <int LANES, bool NORM>
__global__ void __launch_bounds__(kThreads) qk_fwd_kernel(const __grid_constant__ QkParams p) {
  const uint32_t lane = lane_id();
  const int c = static_cast<int>(lane & (LANES - 1));
  const uint32_t mask = row_mask<LANES>(lane);
  const bool on = c < p.d / 8;
  const LaneBlocks blk = lane_blocks(p, on ? c : 0);
  const float inv_d = 1.0f / static_cast<float>(p.d);
  const int groups_q = (p.heads[0] + kFwdHeads - 1) / kFwdHeads;
  const int groups_k = (p.heads[1] + kFwdHeads - 1) / kFwdHeads;
  const int64_t items_q = p.tokens * groups_q;
  const int64_t items = items_q + p.tokens * groups_k;
  const int64_t slots = static_cast<int64_t>(gridDim.x) * (kThreads / LANES);
  for (int64_t u0 = static_cast<int64_t>(blockIdx.x) * (kThreads / LANES) + threadIdx.x / LANES; u0 < items;
       u0 += slots) {
    const int which = u0 >= items_q ? 1 : 0;
    const int64_t u = which ? u0 - items_q : u0;
    const int groups = which ? groups_k : groups_q;
    const int64_t tok = u / groups;
    const int h0 = static_cast<int>(u - tok * groups) * kFwdHeads;
    const int n = min(kFwdHeads, p.heads[which] - h0);
    const uint4* x = static_cast<const uint4*>(p.x[which]) + (tok * p.sx[which].row + h0 * p.sx[which].head) / 8 + c;
    const int64_t xh = p.sx[which].head / 8;
    uint4 v[kFwdHeads];
#pragma unroll
    for (int j = 0; j < kFwdHeads; ++j) v[j] = on && j < n ? x[j * xh] : make_uint4(0u, 0u, 0u, 0u);
    float4 t0, t1;
    block_angles(p, blk, tok, t0, t1);
    if (p.inverse) rope_transpose(t0, t1);
    uint4* y = static_cast<uint4*>(p.y[which]) + (tok * p.sy[which].row + h0 * p.sy[which].head) / 8 + c;
    const int64_t yh = p.sy[which].head / 8;
    float w[8];
    if constexpr (NORM) load_weights(p.g[which], on ? c : 0, w);
#pragma unroll
    for (int j = 0; j < kFwdHeads; ++j) {
      if (j >= n) break;
      uint4 out;
      if constexpr (NORM) {
        float e[8];
        unpack8(v[j], e);
        float sq = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) sq = fmaf(e[k], e[k], sq);
        const float r = rsqrtf(row_sum<LANES>(sq, mask) * inv_d + p.eps);
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] *= r * w[k];
        turn8(e, t0, t1);
        out = pack8(e);
      } else {
        out = rot_bf16x8(v[j], t0, t1);
      }
      if (on) y[j * yh] = out;
    }
  }
}

// Backward.  Work item: a group of up to kBwdHeads heads of one token.  The
// lanes add e o n for their chunk over all their rows; a block then adds its
// rows' shares in a fixed order into partial[which][block][d], and
// qk_dg_kernel adds the blocks', again in a fixed order: no atomics, the
// same bits on every run.
template <int LANES>
__global__ void __launch_bounds__(kThreads) qk_bwd_kernel(const __grid_constant__ QkParams p) {
  constexpr int kRows = kThreads / LANES;
  __shared__ float red[kRows][LANES * 8 + 4];
  const uint32_t lane = lane_id();
  const int c = static_cast<int>(lane & (LANES - 1));
  const uint32_t mask = row_mask<LANES>(lane);
  const bool on = c < p.d / 8;
  const LaneBlocks blk = lane_blocks(p, on ? c : 0);
  const float inv_d = 1.0f / static_cast<float>(p.d);
  const int slot = static_cast<int>(threadIdx.x) / LANES;
  for (int which = 0; which < 2; ++which) {
    if (p.heads[which] == 0) break;
    const int groups = (p.heads[which] + kBwdHeads - 1) / kBwdHeads;
    const int64_t items = p.tokens * groups;
    float w[8], dg[8];
    load_weights(p.g[which], on ? c : 0, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) dg[k] = 0.f;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kRows + slot; u < items;
         u += static_cast<int64_t>(gridDim.x) * kRows) {
      const int64_t tok = u / groups;
      const int h0 = static_cast<int>(u - tok * groups) * kBwdHeads;
      const int n = min(kBwdHeads, p.heads[which] - h0);
      const uint4* x = static_cast<const uint4*>(p.x[which]) + (tok * p.sx[which].row + h0 * p.sx[which].head) / 8 + c;
      const uint4* dy =
          static_cast<const uint4*>(p.dy[which]) + (tok * p.sdy[which].row + h0 * p.sdy[which].head) / 8 + c;
      uint4 v[kBwdHeads], dv[kBwdHeads];
#pragma unroll
      for (int j = 0; j < kBwdHeads; ++j) {
        const bool ld = on && j < n;
        v[j] = ld ? x[j * (p.sx[which].head / 8)] : make_uint4(0u, 0u, 0u, 0u);
        dv[j] = ld ? dy[j * (p.sdy[which].head / 8)] : make_uint4(0u, 0u, 0u, 0u);
      }
      float4 t0, t1;
      block_angles(p, blk, tok, t0, t1);
      rope_transpose(t0, t1);
      uint4* dx = static_cast<uint4*>(p.y[which]) + (tok * p.sy[which].row + h0 * p.sy[which].head) / 8 + c;
#pragma unroll
      for (int j = 0; j < kBwdHeads; ++j) {
        if (j >= n) break;
        float e[8], xv[8];
        unpack8(v[j], xv);
        unpack8(dv[j], e);
        turn8(e, t0, t1);
        float sq = 0.f, tx = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          sq = fmaf(xv[k], xv[k], sq);
          tx = fmaf(e[k] * w[k], xv[k], tx);
        }
        const float r = rsqrtf(row_sum<LANES>(sq, mask) * inv_d + p.eps);
        // mean(t o n) = r mean(t o x), and n = r x.
        const float m = row_sum<LANES>(tx, mask) * inv_d * r;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float nk = xv[k] * r;
          dg[k] = fmaf(e[k], nk, dg[k]);
          e[k] = r * fmaf(-nk, m, e[k] * w[k]);
        }
        if (on) dx[j * (p.sy[which].head / 8)] = pack8(e);
      }
    }
    // The block's share of dg, row by row.
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) red[slot][c * 8 + k] = dg[k];
    __syncthreads();
    for (int k = threadIdx.x; k < p.d; k += kThreads) {
      float s = 0.f;
      for (int i = 0; i < kRows; ++i) s += red[i][k];
      p.partial[(static_cast<int64_t>(which) * gridDim.x + blockIdx.x) * p.d + k] = s;
    }
  }
}

// dg[which][k] = the sum over `blocks` partials; one block per 32 columns of
// one weight vector.
__global__ void __launch_bounds__(1024) qk_dg_kernel(const float* partial, int blocks, int d, float* dgq, float* dgk) {
  __shared__ float red[32][33];
  const int col = static_cast<int>(blockIdx.x) * 32 + (threadIdx.x & 31);
  const int row = threadIdx.x >> 5;
  float* dst = blockIdx.y ? dgk : dgq;
  const float* src = partial + static_cast<int64_t>(blockIdx.y) * blocks * d;
  float s = 0.f;
  if (dst && col < d)
    for (int b = row; b < blocks; b += 32) s += src[static_cast<int64_t>(b) * d + col];
  red[row][threadIdx.x & 31] = s;
  __syncthreads();
  s = red[threadIdx.x & 31][row];     // column `row` of the tile, partial row = lane
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  const int out = static_cast<int>(blockIdx.x) * 32 + row;
  if (dst && (threadIdx.x & 31) == 0 && out < d) dst[out] = s;
}

template <int LANES>
cudaError_t launch_fwd_t(const QkParams& p, bool norm, cudaStream_t stream) {
  const int64_t items = p.tokens * ((p.heads[0] + kFwdHeads - 1) / kFwdHeads + (p.heads[1] + kFwdHeads - 1) / kFwdHeads);
  int64_t blocks = (items * LANES + kThreads - 1) / kThreads;
  if (blocks > 152 * 32) blocks = 152 * 32;
  if (norm) qk_fwd_kernel<LANES, true><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
  else qk_fwd_kernel<LANES, false><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

int qk_bwd_blocks(int64_t tokens, int heads_q, int heads_k, int d) {
  const int rows = kThreads / (d <= 64 ? 8 : 16);
  const int64_t most = tokens * ((std::max(heads_q, heads_k) + kBwdHeads - 1) / kBwdHeads);
  const int64_t blocks = (most + rows - 1) / rows;
  return static_cast<int>(blocks < 152 * 4 ? blocks : 152 * 4);
}

cudaError_t launch_qk_fwd(const QkParams& p, bool norm, cudaStream_t stream) {
  return p.d <= 64 ? launch_fwd_t<8>(p, norm, stream) : launch_fwd_t<16>(p, norm, stream);
}

cudaError_t launch_qk_bwd(const QkParams& p, float* dgq, float* dgk, cudaStream_t stream) {
  const int blocks = qk_bwd_blocks(p.tokens, p.heads[0], p.heads[1], p.d);
  if (p.d <= 64) qk_bwd_kernel<8><<<blocks, kThreads, 0, stream>>>(p);
  else qk_bwd_kernel<16><<<blocks, kThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!dgq && !dgk)) return e;
  qk_dg_kernel<<<dim3((p.d + 31) / 32, 2), 1024, 0, stream>>>(p.partial, blocks, p.d, dgq, dgk);
  return cudaGetLastError();
}

}  // namespace esd
