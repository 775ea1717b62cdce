// act_bwd.cu -- first step of the backward of the experts' products:
// dH = dY act'(H) and the bias gradients sum_r dH_r, one pass over dY and H.
//
// A tile is 64 rows of one expert by 256 columns; 8 row lanes of a block each
// add up their rows in registers, join in shared memory and leave one fp32
// partial per tile and column, which a second kernel adds in the order of the
// tiles (no atomics: the same bits every time).  dH is rounded to the type, in
// which the two products that follow take it; the bias sums add it unrounded.  Bound
// by memory: dY and H in, dH out; the partials are 1/64 of that.  Measured at 16384
// x 4096, bf16, in a graph: relu 67 us (6.0 TB/s), silu 73, gelu 78, swiglu (2 x
// 2048) 54 (6.2); the bias sums add 10 to 12.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "activation.cuh"
#include "chain.cuh"
#include "experts.h"

namespace lapsum {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 64;    // rows per tile
constexpr int kCols = 256;   // columns per tile: 32 threads of 8
constexpr int kMaxTable = LAPSUM_EXPERTS_MAX + 1;

struct ActArgs {
  const uint16_t* gy;
  int64_t gy_stride;
  const uint16_t* h;
  int64_t h_stride;
  uint16_t* gh;
  int64_t gh_stride;
  float* part;  // [tiles][out] or null
  int64_t rows;
  int width;    // columns of dY
  int out;      // columns of dH (2 width when gated)
  int experts, bf16, act;
  const int32_t* offsets;
};

__device__ __forceinline__ void unpack8(const uint4& q, int bf16, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8], int bf16) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      const __half2 b = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// rows [lo, lo + n) of expert e, clamped into the array
__device__ __forceinline__ void range_of(const int32_t* offsets, int64_t rows, int e, int& lo, int& n) {
  if (!offsets) {
    lo = 0;
    n = (int)rows;
    return;
  }
  lo = min(max(__ldg(offsets + e), 0), (int)rows);
  n = max(min(max(__ldg(offsets + e + 1), 0), (int)rows) - lo, 0);
}

// table[e] = row tiles before expert e, table[experts] = all (one warp)
__device__ __forceinline__ void fill_table(const int32_t* offsets, int64_t rows, int experts, int* table, int lane) {
  int base = 0;
  for (int e0 = 0; e0 < experts; e0 += 32) {
    const int e = e0 + lane;
    int lo, n = 0;
    if (e < experts) range_of(offsets, rows, e, lo, n);
    const int own = (n + kRows - 1) / kRows;
    int v = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += u;
    }
    if (e < experts) table[e] = base + v - own;
    base += __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) table[experts] = base;
}

// (four blocks per SM without gates, 86 -> 82 us; with them that would spill)
template <bool kGated>
__global__ void __launch_bounds__(kThreads, kGated ? 1 : 4) k_act_bwd(const ActArgs a, int max_tiles) {
  grid_launch_next();
  grid_wait_previous();
  __shared__ int table[kMaxTable + 1];
  __shared__ float red[2][8][kCols];
  const int col = threadIdx.x & 31, lane8 = threadIdx.x >> 5;
  if (threadIdx.x < 32) fill_table(a.offsets, a.rows, a.experts, table, threadIdx.x);
  __syncthreads();
  const int ctiles = (a.width + kCols - 1) / kCols;
  // the partials hold max_tiles tiles, which ascending offsets never exceed
  const int tiles = min(table[a.experts], max_tiles) * ctiles;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int tt = tile / ctiles, f = (tile - tt * ctiles) * kCols + col * 8;
    int lo = 0, hi = a.experts - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (table[mid] <= tt) lo = mid; else hi = mid - 1;
    }
    int row0, n;
    range_of(a.offsets, a.rows, lo, row0, n);
    const int skip = (tt - table[lo]) * kRows;
    row0 += skip;
    n = min(n - skip, kRows);
    float s0[8] = {}, s1[8] = {};
    if (f < a.width) {
      // four rows of a lane in flight
      for (int r0 = lane8; r0 < n; r0 += 32) {
        uint4 qg[4], qh[4], qu[kGated ? 4 : 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t row = row0 + min(r0 + 8 * i, n - 1);
          qg[i] = __ldg(reinterpret_cast<const uint4*>(a.gy + row * a.gy_stride + f));
          if (kGated || a.act != LAPSUM_ACT_NONE) qh[i] = __ldg(reinterpret_cast<const uint4*>(a.h + row * a.h_stride + f));
          if constexpr (kGated) qu[i] = __ldg(reinterpret_cast<const uint4*>(a.h + row * a.h_stride + a.width + f));
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = r0 + 8 * q;
          if (r >= n) break;
          const int64_t row = row0 + r;
          float g[8], h[8];
          unpack8(qg[q], a.bf16, g);
          if constexpr (kGated) {
            float u[8], d[8];
            unpack8(qh[q], a.bf16, h);
            unpack8(qu[q], a.bf16, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float s = sigmoid_of(h[i]);
              // (factors that vanish first: a large g u must not meet a 0 as infinity)
              d[i] = g[i] * (s * fmaf(h[i], 1.0f - s, 1.0f)) * u[i];
              u[i] = g[i] * (h[i] * s);
              s0[i] += d[i];
              s1[i] += u[i];
            }
            *reinterpret_cast<uint4*>(a.gh + row * a.gh_stride + f) = pack8(d, a.bf16);
            *reinterpret_cast<uint4*>(a.gh + row * a.gh_stride + a.width + f) = pack8(u, a.bf16);
          } else {
            if (a.act != LAPSUM_ACT_NONE) {
              unpack8(qh[q], a.bf16, h);
              differentiate(g, h, a.act);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) s0[i] += g[i];
            if (a.gh) *reinterpret_cast<uint4*>(a.gh + row * a.gh_stride + f) = pack8(g, a.bf16);
          }
        }
      }
    }
    if (a.part) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        red[0][lane8][i * 32 + col] = s0[i];
        if (kGated) red[1][lane8][i * 32 + col] = s1[i];
      }
      __syncthreads();
      const int c = threadIdx.x, at = (tile - tt * ctiles) * kCols + (c & 31) * 8 + (c >> 5);
      if (at < a.width) {
#pragma unroll
        for (int h = 0; h < (kGated ? 2 : 1); ++h) {
          float v = 0.0f;
#pragma unroll
          for (int l = 0; l < 8; ++l) v += red[h][l][c];
          a.part[(int64_t)tt * a.out + h * a.width + at] = v;
        }
      }
    }
  }
}

// grad_bias[e][c] = sum of the expert's partials in the order of its tiles:
// 8 lanes take every 8th tile each, then join in the order of the lanes.
__global__ void __launch_bounds__(kThreads) k_bias_sum(const float* part, int out, int64_t rows, int experts,
                                                       const int32_t* offsets, int max_tiles, int bf16, uint16_t* gb) {
  grid_launch_next();
  grid_wait_previous();
  __shared__ float red[8][32];
  __shared__ int table[kMaxTable + 1];
  const int e = blockIdx.y, c = blockIdx.x * 32 + (threadIdx.x & 31), l = threadIdx.x >> 5;
  if (threadIdx.x < 32) fill_table(offsets, rows, experts, table, threadIdx.x);
  __syncthreads();
  float v = 0.0f;
  if (c < out)
    for (int t = table[e] + l; t < min(table[e + 1], max_tiles); t += 8) v += part[(int64_t)t * out + c];
  red[l][threadIdx.x & 31] = v;
  __syncthreads();
  if (l == 0 && c < out) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += red[i][threadIdx.x];
    gb[(int64_t)e * out + c] = bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
  }
}

int64_t tile_bound(int64_t rows, int experts) { return std::min<int64_t>(experts, rows) + rows / kRows; }

}  // namespace

size_t act_bwd_workspace(int64_t rows, int experts, int64_t out) {
  return ((size_t)tile_bound(rows, experts) * (size_t)out * 4 + 255) & ~size_t(255);
}

cudaError_t launch_act_bwd(const void* grad_y, int bf16, int64_t rows, int64_t out, int64_t grad_y_stride,
                           const void* preact, int64_t preact_stride, int experts, const int32_t* offsets,
                           int activation, void* grad_h, int64_t grad_h_stride, void* grad_bias, void* ws, int sms,
                           cudaStream_t st) {
  const bool gated = activation == LAPSUM_ACT_SWIGLU;
  ActArgs a{};
  a.gy = static_cast<const uint16_t*>(grad_y);
  a.gy_stride = grad_y_stride;
  a.h = static_cast<const uint16_t*>(preact);
  a.h_stride = preact_stride;
  a.gh = static_cast<uint16_t*>(grad_h);
  a.gh_stride = grad_h_stride;
  a.part = grad_bias ? static_cast<float*>(ws) : nullptr;
  a.rows = rows;
  a.out = (int)out;
  a.width = (int)(gated ? out / 2 : out);
  a.experts = experts;
  a.bf16 = bf16;
  a.act = activation;
  a.offsets = offsets;
  const int64_t bound = tile_bound(rows, experts);
  const int64_t grid = std::min<int64_t>(bound * ((a.width + kCols - 1) / kCols), (int64_t)sms * 6);
  {
    Launch guard("k_act_bwd", st);
    if (gated)
      launch_ex(true, k_act_bwd<true>, dim3((unsigned)grid), dim3(kThreads), 0, st, a, (int)bound);
    else
      launch_ex(true, k_act_bwd<false>, dim3((unsigned)grid), dim3(kThreads), 0, st, a, (int)bound);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !grad_bias) return e;
  Launch guard("k_bias_sum", st);
  launch_ex(true, k_bias_sum, dim3((unsigned)((out + 31) / 32), (unsigned)experts), dim3(kThreads), 0, st,
      a.part, a.out, rows, experts, offsets, (int)bound, bf16, static_cast<uint16_t*>(grad_bias));
  return cudaGetLastError();
}

}  // namespace lapsum
