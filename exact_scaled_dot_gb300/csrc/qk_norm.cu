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
// and out), 6 backward (x and dy in, dx out), and are bound by DRAM (of the
// measured copy rate: norm and rotation of 8192 tokens of 32 + 8 heads of 128
// in 27 us, 92 %; the backward of 32768 tokens in 160 us, 94 %; the rotation of
// 65537 tokens of 16 + 16 heads in 156 us, 103 %).  Eight
// lanes hold a row, each one or two chunks of 8 elements (16-byte accesses;
// up to width 64, up to 128), and sum over it with three shuffles.  Lanes
// walk over the heads of a token, so that the token's angles (and with them
// the products of cosines, sines and weights) are formed once for up to
// kMostHeads rows, and request several rows before they work on the first.
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "ptx.cuh"
#include "rotary.cuh"

namespace esd {
namespace {

constexpr int kThreads = 128;
constexpr int kLanes = 8;                      // lanes of a row
constexpr int kSlots = kThreads / kLanes;      // tokens that a block works on at once
// Heads of one token that a slot takes, at most.  More share the angles,
// fewer balance the blocks: forward 27.5, 26.9, 28.2 us with 8, 16, 32 heads
// (8192 tokens, 32 + 8 heads of 128), backward 160, 164 us with 8, 16 (32768).
constexpr int kFwdHeads = 16;
constexpr int kBwdHeads = 8;
constexpr int kStages = 4;                     // steps in the ring (a power of two)
constexpr int kBwdResident = 4;                // backward blocks of an SM (128 registers a thread)

// Over the eight lanes of a row; called by whole warps.
__device__ __forceinline__ float row_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  return v + __shfl_xor_sync(0xffffffffu, v, 4);
}

// 1 / sqrt(x) of a normal positive x (x >= eps), to a few 1e-7.
__device__ __forceinline__ float inv_sqrt(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
  x[0] = bf16_lo(v.x), x[1] = bf16_hi(v.x), x[2] = bf16_lo(v.y), x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z), x[5] = bf16_hi(v.z), x[6] = bf16_lo(v.w), x[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// 16 bytes from global to shared memory, in the thread's current group.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {      // all but the last N groups are there
  asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

// Which heads of which tensor a block works on: blockIdx.y counts the parts
// of the query heads, then those of the key heads.
struct Part {
  int which, h0, n;
};
__device__ __forceinline__ Part part_of(const QkParams& p) {
  const int y = static_cast<int>(blockIdx.y);
  const int which = y >= p.parts_q ? 1 : 0;
  const int h0 = (which ? y - p.parts_q : y) * p.part_heads;
  return Part{which, h0, min(p.part_heads, p.heads[which] - h0)};
}

// The frequencies (hi, lo) of every block, in shared memory: read once per token
// by lanes that differ in the block.  (Lanes that differ read a kernel's
// parameters one after the other: one read each, of the blocks there are.  Three
// reads each, of 64 blocks, and ahead of the rows: 8 tokens 2.8 us instead of
// 2.5, 1025 of 16 + 2 heads 4.3 instead of 3.5.)
struct BlockTable {
  float2 w[64];
};
__device__ __forceinline__ void fill_table(const QkParams& p, BlockTable& t) {
  const int k = static_cast<int>(threadIdx.x);
  if (p.axes > 0 && k < p.d / 2) t.w[k] = p.w[k];
  __syncthreads();
}

// The axes of the four blocks of chunk c, a byte each: kept where angles are
// formed in a loop.
__device__ __forceinline__ uint32_t chunk_axes(const QkParams& p, int c) {
  uint32_t axes = 0u;
#pragma unroll
  for (int q = 0; q < 4; ++q) axes |= ((4 * c + q >= p.first[1] ? 1u : 0u) + (4 * c + q >= p.first[2] ? 1u : 0u)) << (8 * q);
  return axes;
}

// Cosines and sines of the four blocks of chunk c at the token's positions
// (the same angles as the single-axis rotation); t0: blocks 0, 1, t1: 2, 3.
// position(q): the position that the chunk's block q turns by.
template <class Position>
__device__ __forceinline__ void chunk_angles(const QkParams& p, const BlockTable& tab, Position position, int c,
                                             float4& t0, float4& t1) {
  if (p.axes == 0) {
    t0 = t1 = make_float4(1.f, 0.f, 1.f, 0.f);
    return;
  }
  float cs[4], sn[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float2 w = tab.w[4 * c + q];
    rope_cos_sin(reduced_angle(position(q), w.x, w.y), cs[q], sn[q]);
  }
  t0 = make_float4(cs[0], sn[0], cs[1], sn[1]);
  t1 = make_float4(cs[2], sn[2], cs[3], sn[3]);
}

__device__ __forceinline__ void token_positions(const QkParams& p, int64_t tok, int32_t (&pos)[kMaxAxes]) {
#pragma unroll
  for (int a = 0; a < kMaxAxes; ++a) pos[a] = a < p.axes ? p.pos[a * p.tokens + tok] : 0;
}

// Weights of chunk c (ones without a weight vector).
__device__ __forceinline__ void load_weights(const void* g, int c, float (&w)[8]) {
  if (g) {
    unpack8(static_cast<const uint4*>(g)[c], w);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = 1.f;
  }
}

// Forward.  CH chunks per lane: chunk i of lane c is c + 8 i.
template <int CH, bool NORM>
__global__ void __launch_bounds__(kThreads) qk_fwd_kernel(const __grid_constant__ QkParams p) {
  constexpr int kRows = CH == 1 ? 4 : 2;       // rows of a step
  __shared__ BlockTable tab;
  __shared__ uint4 ring[kStages][kRows * CH][kThreads];
  const uint32_t lane = lane_id();
  const int c = static_cast<int>(lane & 7);
  const Part part = part_of(p);
  const float inv_d = 1.0f / static_cast<float>(p.d);
  // Slots past the last token go along with the last one and write nothing.
  const int64_t slot_tok = static_cast<int64_t>(blockIdx.x) * kSlots + threadIdx.x / kLanes;
  const bool there = slot_tok < p.tokens;
  const int64_t tok = there ? slot_tok : p.tokens - 1;
  const int64_t xh = p.sx[part.which].head / 8, yh = p.sy[part.which].head / 8;
  const uint4* x = static_cast<const uint4*>(p.x[part.which]) + tok * (p.sx[part.which].row / 8) + part.h0 * xh + c;
  uint4* y = static_cast<uint4*>(p.y[part.which]) + tok * (p.sy[part.which].row / 8) + part.h0 * yh + c;
  bool on[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) on[i] = c + 8 * i < p.d / 8;
  auto request = [&](int it) {       // the rows of step `it`
    const int h = it * kRows;
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (on[i] && h + j < part.n)
          copy16(smem_u32(&ring[it & (kStages - 1)][j * CH + i][threadIdx.x]), x + (h + j) * xh + 8 * i);
    copy_commit();
  };
#pragma unroll
  for (int it = 0; it < kStages - 1; ++it) request(it);
  int32_t pos[kMaxAxes];
  token_positions(p, tok, pos);
  fill_table(p, tab);        // behind the first requests
  // cs: the cosines and sines; with a norm, each block's map (x0, x1) ->
  // (x0 a - x1 b, x0 c + x1 d) with the weights in it.
  float4 cs[CH][2], map[CH][4];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int ci = on[i] ? c + 8 * i : 0;
    chunk_angles(p, tab, [&](int q) {
      const int k = 4 * ci + q;
      return k < p.first[1] ? pos[0] : (k < p.first[2] ? pos[1] : pos[2]);
    }, ci, cs[i][0], cs[i][1]);
    if (p.inverse) rope_transpose(cs[i][0], cs[i][1]);
    if constexpr (NORM) {
      float w[8];
      load_weights(p.g[part.which], ci, w);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 t = cs[i][q / 2];
        const float co = q & 1 ? t.z : t.x, si = q & 1 ? t.w : t.y;
        map[i][q] = make_float4(w[2 * q] * co, w[2 * q + 1] * si, w[2 * q] * si, w[2 * q + 1] * co);
      }
    }
  }
  for (int it = 0; it * kRows < part.n; ++it) {
    copy_wait<kStages - 2>();
    uint4 v[kRows][CH];
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        v[j][i] = ring[it & (kStages - 1)][j * CH + i][threadIdx.x];
        if (!on[i]) v[j][i] = make_uint4(0u, 0u, 0u, 0u);
      }
    request(it + kStages - 1);
    const int h = it * kRows;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if constexpr (NORM) {
        float e[CH][8], sq = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          unpack8(v[j][i], e[i]);
#pragma unroll
          for (int k = 0; k < 8; ++k) sq = fmaf(e[i][k], e[i][k], sq);
        }
        const float r = inv_sqrt(fmaf(row_sum(sq), inv_d, p.eps));
#pragma unroll
        for (int i = 0; i < CH; ++i) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float x0 = e[i][2 * q], x1 = e[i][2 * q + 1];
            e[i][2 * q] = r * fmaf(x0, map[i][q].x, -(x1 * map[i][q].y));
            e[i][2 * q + 1] = r * fmaf(x0, map[i][q].z, x1 * map[i][q].w);
          }
          if (there && on[i] && h + j < part.n) y[(h + j) * yh + 8 * i] = pack8(e[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < CH; ++i)
          if (there && on[i] && h + j < part.n) y[(h + j) * yh + 8 * i] = rot_bf16x8(v[j][i], cs[i][0], cs[i][1]);
      }
    }
  }
  copy_wait<0>();        // (only empty groups are left)
}

// Steps of the backward's lanes: kRows heads of one token after another, then the next
// token.  A cursor names a step; the ring's runs kStages - 1 steps ahead.
template <int ROWS>
struct Cursor {
  int64_t tok;
  int h;
  __device__ __forceinline__ void next(int n, int64_t step) {
    h += ROWS;
    if (h >= n) {
      h = 0;
      tok += step;
    }
  }
};

// Backward.  The lanes add e o n for their chunks over all their rows; a
// block then adds its slots' shares in a fixed order into
// partial[blockIdx.y][blockIdx.x][d], and qk_dg_kernel adds the blocks', again
// in a fixed order: no atomics, the same bits on every run.
template <int CH>
__global__ void __launch_bounds__(kThreads, kBwdResident) qk_bwd_kernel(const __grid_constant__ QkParams p) {
  constexpr int kRows = CH == 1 ? 2 : 1;       // rows of a step
  __shared__ BlockTable tab;
  // The ring (x, then dy), and at the end the slots' shares of dg.
  __shared__ union {
    uint4 ring[kStages][2][kRows * CH][kThreads];
    float red[kSlots][CH * 64 + 4];
  } sh;
  const uint32_t lane = lane_id();
  const int c = static_cast<int>(lane & 7);
  const Part part = part_of(p);
  const float inv_d = 1.0f / static_cast<float>(p.d);
  const int64_t xr = p.sx[part.which].row / 8, xh = p.sx[part.which].head / 8;
  const int64_t dyr = p.sdy[part.which].row / 8, dyh = p.sdy[part.which].head / 8;
  const int64_t dxr = p.sy[part.which].row / 8, dxh = p.sy[part.which].head / 8;
  const uint4* x = static_cast<const uint4*>(p.x[part.which]) + part.h0 * xh + c;
  const uint4* dy = static_cast<const uint4*>(p.dy[part.which]) + part.h0 * dyh + c;
  uint4* dx = static_cast<uint4*>(p.y[part.which]) + part.h0 * dxh + c;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kSlots;
  // The warps go through the steps together: the block's first slot decides.
  Cursor<kRows> at{static_cast<int64_t>(blockIdx.x) * kSlots + threadIdx.x / kLanes, 0}, ahead = at;
  const int slot = static_cast<int>(threadIdx.x) / kLanes;
  bool on[CH];
  float w[CH][8], dg[CH][8];
  uint32_t axes[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    on[i] = c + 8 * i < p.d / 8;
    axes[i] = chunk_axes(p, c + 8 * i);
    load_weights(p.g[part.which], on[i] ? c + 8 * i : 0, w[i]);
#pragma unroll
    for (int k = 0; k < 8; ++k) dg[i][k] = 0.f;
  }
  auto request = [&](int stage) {
    if (ahead.tok < p.tokens) {
      const uint4* rx = x + ahead.tok * xr + ahead.h * xh;
      const uint4* rd = dy + ahead.tok * dyr + ahead.h * dyh;
#pragma unroll
      for (int j = 0; j < kRows; ++j)
#pragma unroll
        for (int i = 0; i < CH; ++i)
          if (on[i] && ahead.h + j < part.n) {
            copy16(smem_u32(&sh.ring[stage][0][j * CH + i][threadIdx.x]), rx + j * xh + 8 * i);
            copy16(smem_u32(&sh.ring[stage][1][j * CH + i][threadIdx.x]), rd + j * dyh + 8 * i);
          }
    }
    copy_commit();
    ahead.next(part.n, step);
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) request(s);
  float4 cs[CH][2];
#pragma unroll
  for (int i = 0; i < CH; ++i) cs[i][0] = cs[i][1] = make_float4(1.f, 0.f, 1.f, 0.f);    // (slots without a token)
  int32_t pos[kMaxAxes];
  if (at.tok < p.tokens) token_positions(p, at.tok, pos);
  fill_table(p, tab);        // behind the first requests
  for (int it = 0; at.tok - slot < p.tokens; ++it) {
    const bool there = at.tok < p.tokens;
    if (at.h == 0 && there) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        chunk_angles(p, tab, [&](int q) {
          const uint32_t axis = axes[i] >> (8 * q) & 0xFFu;
          return axis == 0u ? pos[0] : (axis == 1u ? pos[1] : pos[2]);
        }, on[i] ? c + 8 * i : 0, cs[i][0], cs[i][1]);
        rope_transpose(cs[i][0], cs[i][1]);
      }
      if (at.tok + step < p.tokens) token_positions(p, at.tok + step, pos);     // the next token's, early
    }
    copy_wait<kStages - 2>();
    const int stage = it & (kStages - 1);
    uint4 v[kRows][CH], dv[kRows][CH];
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const bool read = there && on[i] && at.h + j < part.n;
        v[j][i] = sh.ring[stage][0][j * CH + i][threadIdx.x];
        dv[j][i] = sh.ring[stage][1][j * CH + i][threadIdx.x];
        if (!read) v[j][i] = dv[j][i] = make_uint4(0u, 0u, 0u, 0u);
      }
    request((it + kStages - 1) & (kStages - 1));
    uint4* row = dx + at.tok * dxr + at.h * dxh;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      float e[CH][8], xv[CH][8], pr[CH][8], sq = 0.f, tx = 0.f;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        unpack8(v[j][i], xv[i]);
        unpack8(dv[j][i], e[i]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 t = cs[i][q / 2];
          float y0, y1;
          rot_block(e[i][2 * q], e[i][2 * q + 1], q & 1 ? t.z : t.x, q & 1 ? t.w : t.y, y0, y1);
          e[i][2 * q] = y0;
          e[i][2 * q + 1] = y1;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          sq = fmaf(xv[i][k], xv[i][k], sq);
          pr[i][k] = e[i][k] * xv[i][k];
          tx = fmaf(w[i][k], pr[i][k], tx);            // t o x = g o e o x
        }
      }
      const float r = inv_sqrt(fmaf(row_sum(sq), inv_d, p.eps));
      const float m = row_sum(tx) * inv_d * r * r;          // dx = r (t - m x); r^3 may pass fp32's range
#pragma unroll
      for (int i = 0; i < CH; ++i) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          dg[i][k] = fmaf(r, pr[i][k], dg[i][k]);
          e[i][k] = r * fmaf(w[i][k], e[i][k], -(m * xv[i][k]));
        }
        if (there && on[i] && at.h + j < part.n) row[j * dxh + 8 * i] = pack8(e[i]);
      }
    }
    at.next(part.n, step);
  }
  copy_wait<0>();        // (only empty groups are left)
  __syncthreads();
  // The block's share of dg, slot by slot.
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) sh.red[threadIdx.x / kLanes][(c + 8 * i) * 8 + k] = dg[i][k];
  __syncthreads();
  for (int k = threadIdx.x; k < p.d; k += kThreads) {
    float s = 0.f;
    for (int i = 0; i < kSlots; ++i) s += sh.red[i][k];
    p.partial[(static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * p.d + k] = s;
  }
}

// dgq and dgk: the sums over their blocks' partials (the first blocks_q,
// then the rest); one block per 32 columns of one weight vector.
__global__ void __launch_bounds__(1024) qk_dg_kernel(const float* partial, int blocks_q, int blocks_k, int d, float* dgq,
                                                     float* dgk) {
  __shared__ float red[32][33];
  const int col = static_cast<int>(blockIdx.x) * 32 + (threadIdx.x & 31);
  const int row = threadIdx.x >> 5;
  float* dst = blockIdx.y ? dgk : dgq;
  const float* src = partial + (blockIdx.y ? static_cast<int64_t>(blocks_q) * d : 0);
  const int blocks = blockIdx.y ? blocks_k : blocks_q;
  cudaGridDependencySynchronize();
  float s = 0.f;
  if (dst && col < d) {
#pragma unroll 4
    for (int b = row; b < blocks; b += 32) s += src[static_cast<int64_t>(b) * d + col];
  }
  red[row][threadIdx.x & 31] = s;
  __syncthreads();
  s = red[threadIdx.x & 31][row];     // column `row` of the tile, partial row = lane
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  const int out = static_cast<int>(blockIdx.x) * 32 + row;
  if (dst && (threadIdx.x & 31) == 0 && out < d) dst[out] = s;
}

int parts_of(int heads, int part_heads) { return (heads + part_heads - 1) / part_heads; }

// Heads that a slot takes: `most`, fewer while the blocks would leave SMs
// idle (a decode step's few tokens).
int choose_part_heads(int64_t tokens, int heads_q, int heads_k, int most) {
  int n = most;
  const int64_t rows = (tokens + kSlots - 1) / kSlots;
  while (n > 1 && rows * (parts_of(heads_q, n) + parts_of(heads_k, n)) < 2 * 152) n /= 2;
  return n;
}

// The backward's blocks along the tokens: as many of all parts as are resident,
// so that each works to the end with its ring filled and has one share of dg.
int bwd_blocks_x(int64_t tokens, int parts) {
  const int64_t rows = (tokens + kSlots - 1) / kSlots, most = std::max(1, 152 * kBwdResident / parts);
  return static_cast<int>(std::min(rows, most));
}

}  // namespace

int qk_bwd_blocks(int64_t tokens, int heads_q, int heads_k) {
  const int n = choose_part_heads(tokens, heads_q, heads_k, kBwdHeads);
  const int parts = parts_of(heads_q, n) + parts_of(heads_k, n);
  return parts * bwd_blocks_x(tokens, parts);
}

cudaError_t launch_qk_fwd(QkParams p, bool norm, cudaStream_t stream) {
  p.part_heads = choose_part_heads(p.tokens, p.heads[0], p.heads[1], kFwdHeads);
  p.parts_q = parts_of(p.heads[0], p.part_heads);
  const dim3 grid(static_cast<unsigned>((p.tokens + kSlots - 1) / kSlots),
                  static_cast<unsigned>(p.parts_q + parts_of(p.heads[1], p.part_heads)));
  if (p.d <= 64) {
    if (norm) qk_fwd_kernel<1, true><<<grid, kThreads, 0, stream>>>(p);
    else qk_fwd_kernel<1, false><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (norm) qk_fwd_kernel<2, true><<<grid, kThreads, 0, stream>>>(p);
    else qk_fwd_kernel<2, false><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_qk_bwd(QkParams p, float* dgq, float* dgk, cudaStream_t stream) {
  p.part_heads = choose_part_heads(p.tokens, p.heads[0], p.heads[1], kBwdHeads);
  p.parts_q = parts_of(p.heads[0], p.part_heads);
  const int parts = p.parts_q + parts_of(p.heads[1], p.part_heads);
  const dim3 grid(static_cast<unsigned>(bwd_blocks_x(p.tokens, parts)), static_cast<unsigned>(parts));
  if (p.d <= 64) qk_bwd_kernel<1><<<grid, kThreads, 0, stream>>>(p);
  else qk_bwd_kernel<2><<<grid, kThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!dgq && !dgk)) return e;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((p.d + 31) / 32), 2);
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qk_dg_kernel, static_cast<const float*>(p.partial),
                            static_cast<int>(grid.x) * p.parts_q, static_cast<int>(grid.x) * (parts - p.parts_q), p.d,
                            dgq, dgk);
}

}  // namespace esd
