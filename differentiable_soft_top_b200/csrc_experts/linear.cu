// linear.cu -- the experts' products and their gradients on the tensor cores.
//
// y_r = act(W_e x_r + b_e) + residual_r for the rows of expert e.  Rows are
// few or many per expert and start anywhere, the features of a weight matrix
// are many and regular; so the weights take the fixed side of the matrix
// instruction (M = 128 of its rows) and the tokens the variable one (N = 16 ..
// 256 in steps of 16): D^T = W X^T.  A tile with 5 tokens then costs an N = 16
// instruction, not a 128-row one, and one kernel serves one token and long
// prompts.
//
//   forward          D[f, t] = sum_k W[f, k] X[t, k]       both K major
//   input gradient   D[k, t] = sum_n W[n, k] dH[t, n]      W MN major
//   weight gradient  D[n, k] = sum_t dH[t, n] X[t, k]      both MN major; the
//                    contraction runs over an expert's rows and its ragged
//                    end is zeroed in shared memory
//
// One block of six warps: warp 0 fills a ring of stages by tiled copies (64
// deep, 128-byte swizzle), warp 1 issues the products, warps 2-5 read the
// accumulators from tensor memory (lane = feature) and write the result.  Two
// accumulators let the epilogue of one tile run beside the products of the
// next; blocks walk the tiles with a stride of the grid.  Few rows: one tile
// per cluster of 1, 2, 4 or 8 blocks, which split the contraction and join
// their fp32 partials through distributed shared memory in the order of rank.
//
// Every wait is bounded: a block that gives up sets a status bit, writes NaN
// for what it leaves undone, lets its copies land and frees its tensor memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "experts.h"
#include "umma.cuh"

namespace lapsum {
namespace {

enum Mode { kForward, kGradX, kGradW };

constexpr int kThreads = 192;
constexpr int kDepth = 64;              // contraction per stage: one 128-byte line
constexpr int kFeat = 128;              // features per tile
constexpr int kTokBox = 32;             // tokens per copied box
constexpr uint32_t kPolls = 1u << 22;   // polls of a bounded wait, about a second

struct Args {
  int64_t rows;
  int experts, bf16, activation;
  int feat;          // features of the output (half of the weights' rows when gated)
  int depth;         // contraction length (rows of an expert in kGradW)
  int cols;          // kGradW: columns of the weight gradient
  const int32_t* offsets;
  const void* bias;
  const void* residual;
  int64_t residual_stride;
  void* y;
  int64_t y_stride;
  void* preact;
  int64_t preact_stride;
  uint32_t* status;
};

template <int kMode, int kTok, bool kGated>
struct Shape {
  static constexpr int kABytes = kFeat * 128 * (kGated ? 2 : 1);
  static constexpr int kBBytes = kTok * 128;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr bool kSplit = kTok == 32;  // few rows: clusters, two blocks per SM when ungated
  static constexpr int kBudget = kSplit && !kGated ? 106 * 1024 : 200 * 1024;
  static constexpr int kStages = kBudget / kStage;
  static constexpr int kAccCols = kTok * (kGated ? 2 : 1);
  static constexpr int kTmemCols = kSplit ? (kAccCols < 32 ? 32 : kAccCols) : 2 * kAccCols;
  static constexpr int kTable = kMode == kGradW ? 0 : (LAPSUM_EXPERTS_MAX + 2) * 4;
  static constexpr int kSmem = kStages * kStage + kTable + 1024 /* alignment */ + 512 /* barriers */;
};

__device__ __forceinline__ float load16(const void* p, int64_t i, int bf16) {
  const uint16_t u = __ldg(static_cast<const uint16_t*>(p) + i);
  return bf16 ? __uint_as_float((uint32_t)u << 16) : __half2float(__ushort_as_half(u));
}
__device__ __forceinline__ uint16_t pack16(float v, int bf16) {
  return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}
__device__ __forceinline__ uint32_t pack32(float lo, float hi, int bf16) {
  return (uint32_t)pack16(lo, bf16) | ((uint32_t)pack16(hi, bf16) << 16);
}

__device__ __forceinline__ float sigmoid_of(float h) { return __fdividef(1.0f, 1.0f + __expf(-h)); }

// v = act(v) for the ungated activations
__device__ __forceinline__ void activate(float (&v)[32], int act) {
  if (act == LAPSUM_ACT_RELU) {
#pragma unroll
    for (int c = 0; c < 32; ++c) v[c] = v[c] < 0.0f ? 0.0f : v[c];  // keeps NaN
  } else if (act == LAPSUM_ACT_SILU) {
#pragma unroll
    for (int c = 0; c < 32; ++c) v[c] *= sigmoid_of(v[c]);
  } else if (act == LAPSUM_ACT_GELU) {
#pragma unroll
    for (int c = 0; c < 32; ++c) v[c] *= fmaf(0.5f, erff(v[c] * 0.70710678f), 0.5f);
  }
}

struct Tile {
  int expert;
  int row0, n;   // tokens [row0, row0 + n) (kGradW: the expert's rows)
  int f0;        // first feature
  int c0;        // kGradW: first column
  int chunks;    // stages of this tile's contraction (0: nothing to multiply)
};

// Row range of expert e, clamped into the array whatever the offsets hold;
// "expert" a.experts is the rows behind the last one's.
__device__ __forceinline__ void row_range(const Args& a, int e, int& lo, int& n) {
  const int rows = (int)a.rows;
  int hi = rows;
  if (a.offsets) {
    lo = min(max(__ldg(a.offsets + e), 0), rows);
    if (e < a.experts) hi = min(max(__ldg(a.offsets + e + 1), 0), rows);
  } else {
    lo = e ? rows : 0;
  }
  n = max(hi - lo, 0);
}

// Token tiles before each expert, in shared memory: table[e] for e = 0 ..
// experts + 1 (one warp).
template <int kTok>
__device__ __forceinline__ void build_table(const Args& a, int* table, int lane) {
  int base = 0;
  for (int e0 = 0; e0 <= a.experts; e0 += 32) {
    const int e = e0 + lane;
    int lo = 0, n = 0;
    if (e <= a.experts) row_range(a, e, lo, n);
    int v = (n + kTok - 1) / kTok;
    const int own = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += u;
    }
    if (e <= a.experts) table[e] = base + v - own;
    base += __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) table[a.experts + 1] = base;
}

template <int kMode, int kTok>
__device__ __forceinline__ Tile tile_of(const Args& a, const int* table, int tile) {
  Tile t;
  const int ftiles = (a.feat + kFeat - 1) / kFeat;
  t.c0 = 0;
  if (kMode == kGradW) {
    const int ctiles = (a.cols + kTok - 1) / kTok;
    t.expert = tile / (ftiles * ctiles);
    const int in = tile - t.expert * (ftiles * ctiles);
    t.f0 = (in / ctiles) * kFeat;
    t.c0 = (in % ctiles) * kTok;
    row_range(a, t.expert, t.row0, t.n);
    t.chunks = (t.n + kDepth - 1) / kDepth;
    return t;
  }
  const int tt = tile / ftiles;
  t.f0 = (tile - tt * ftiles) * kFeat;
  int lo = 0, hi = a.experts;  // the last expert whose first tile is <= tt
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (table[mid] <= tt) lo = mid; else hi = mid - 1;
  }
  t.expert = lo;
  int row0, n;
  row_range(a, lo, row0, n);
  const int skip = (tt - table[lo]) * kTok;
  t.row0 = row0 + skip;
  t.n = min(n - skip, kTok);
  t.chunks = lo < a.experts ? (a.depth + kDepth - 1) / kDepth : 0;
  return t;
}


// Bounded wait; a block that has given up somewhere gives up everywhere.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile uint32_t* gave_up) {
  for (uint32_t i = 0; i < kPolls; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 63u && *gave_up) return false;
  }
  *gave_up = 1u;
  return false;
}
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile uint32_t* gave_up) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, gave_up);
}

// 32 tokens of one feature (lane): bias, activation, residual, store.  `up`
// holds the second half's sums of a gated product.
// Of the tile's tokens c0 .. c0 + 31 only those with c % ranks == rank are this
// block's to write.
template <bool kGated>
__device__ __forceinline__ void finish32(const Args& a, const Tile& t, int c0, int f, float b0, float b1,
                                         float (&v)[32], float (&up)[kGated ? 32 : 1], int rank, int ranks) {
  const int m = min(32, t.n - c0);
  const uint32_t own = ranks == 8 ? 0x01010101u << rank : ranks == 4 ? 0x11111111u << rank
                     : ranks == 2 ? 0x55555555u << rank : 0xffffffffu;
  const uint32_t todo = own & (m >= 32 ? 0xffffffffu : (1u << m) - 1u);
  const int64_t row = t.row0 + c0;
  const bool multiplied = t.expert < a.experts;
  if (multiplied) {
#pragma unroll
    for (int c = 0; c < 32; ++c) v[c] += b0;
    if (kGated) {
#pragma unroll
      for (int c = 0; c < 32; ++c) up[c] += b1;
    }
    if (a.preact) {
      uint16_t* h = static_cast<uint16_t*>(a.preact) + row * a.preact_stride + f;
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (todo >> c & 1u) {
          h[c * a.preact_stride] = pack16(v[c], a.bf16);
          if (kGated) h[c * a.preact_stride + a.feat] = pack16(up[c], a.bf16);
        }
    }
    if (kGated) {
#pragma unroll
      for (int c = 0; c < 32; ++c) v[c] *= sigmoid_of(v[c]) * up[c];
    } else {
      activate(v, a.activation);
    }
  } else {
#pragma unroll
    for (int c = 0; c < 32; ++c) v[c] = 0.0f;
  }
  if (a.residual) {
    const int64_t at = row * a.residual_stride + f;
    float r[32];
#pragma unroll
    for (int c = 0; c < 32; ++c) r[c] = (todo >> c & 1u) ? load16(a.residual, at + c * a.residual_stride, a.bf16) : 0.0f;
#pragma unroll
    for (int c = 0; c < 32; ++c) v[c] += r[c];
  }
  uint16_t* y = static_cast<uint16_t*>(a.y) + row * a.y_stride + f;
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (todo >> c & 1u) y[c * a.y_stride] = pack16(v[c], a.bf16);
}

// 32 columns of one row of a weight gradient (both multiples of 8)
__device__ __forceinline__ void store_row32(const Args& a, const Tile& t, int c0, int f, const float (&v)[32]) {
  uint16_t* y = static_cast<uint16_t*>(a.y) + ((int64_t)t.expert * a.feat + f) * a.cols + t.c0 + c0;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (t.c0 + c0 + 8 * q < a.cols) {
      uint4 w;
      w.x = pack32(v[8 * q + 0], v[8 * q + 1], a.bf16);
      w.y = pack32(v[8 * q + 2], v[8 * q + 3], a.bf16);
      w.z = pack32(v[8 * q + 4], v[8 * q + 5], a.bf16);
      w.w = pack32(v[8 * q + 6], v[8 * q + 7], a.bf16);
      *reinterpret_cast<uint4*>(y + 8 * q) = w;
    }
}

// map_f: the weights (kGradW: dH); map_t: the tokens' rows
template <int kMode, int kTok, bool kGated>
__global__ void __launch_bounds__(kThreads, 1)
    k_product(const __grid_constant__ CUtensorMap map_f, const __grid_constant__ CUtensorMap map_t, const Args a,
              int tiles_grad_w) {
  using S = Shape<kMode, kTok, kGated>;
  constexpr int kStages = S::kStages;
  extern __shared__ unsigned char smem_raw[];
  // operands in the 128-byte swizzle start on 1024-byte boundaries
  unsigned char* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char* tail = ring + kStages * S::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(tail);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;    // [2]
  uint64_t* drained = acc_empty + 2;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(drained + 1);
  volatile uint32_t* gave_up = tmem_at + 1;
  int* table = reinterpret_cast<int*>(tail + 512);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    prefetch_map(&map_f);
    prefetch_map(&map_t);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + b, 1);
      mbar_init(acc_empty + b, 4);
    }
    mbar_init(drained, 1);
    *gave_up = 0u;
  }
  if (warp == 1) tmem_alloc(tmem_at, S::kTmemCols);
  if (kMode != kGradW && warp == 2) build_table<kTok>(a, table, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;

  const int ftiles = (a.feat + kFeat - 1) / kFeat;
  const int tiles = kMode == kGradW ? tiles_grad_w : table[a.experts + 1] * ftiles;
  const int ranks = S::kSplit ? (int)cluster_size() : 1;
  const int rank = S::kSplit ? (int)cluster_rank() : 0;
  // few rows: the grid holds a cluster for every tile there can be
  const int first = (int)blockIdx.x / ranks, step = S::kSplit ? max(tiles, 1) : (int)gridDim.x;

  // this block's share of a tile's contraction
  auto share = [&](const Tile& t, int& c0, int& c1) {
    const int per = (t.chunks + ranks - 1) / ranks;
    c0 = min(rank * per, t.chunks);
    c1 = min(c0 + per, t.chunks);
  };

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int tile = first; ok && tile < tiles; tile += step) {
        const Tile t = tile_of<kMode, kTok>(a, table, tile);
        int c0, c1;
        share(t, c0, c1);
        const int boxes = kMode == kGradW ? (min(kTok, a.cols - t.c0) + 63) / 64 : (t.n + kTokBox - 1) / kTokBox;
        const uint32_t bytes = S::kABytes + boxes * (kMode == kGradW ? 8192 : kTokBox * 128);
        for (int c = c0; c < c1; ++c, ++it) {
          const uint32_t s = it % kStages, ph = (it / kStages) & 1u;
          if (!wait_for(empty + s, ph ^ 1u, gave_up)) {
            ok = false;
            break;
          }
          unsigned char* sa = ring + s * S::kStage;
          unsigned char* sb = sa + S::kABytes;
          const int d = c * kDepth;
          mbar_arrive_expect_tx(full + s, bytes);
          if (kMode == kForward) {
            tma_load_3d(sa, &map_f, d, t.f0, t.expert, full + s);
            if (kGated) tma_load_3d(sa + 16384, &map_f, d, a.feat + t.f0, t.expert, full + s);
          } else if (kMode == kGradX) {
            tma_load_3d(sa, &map_f, t.f0, d, t.expert, full + s);
            tma_load_3d(sa + 8192, &map_f, t.f0 + 64, d, t.expert, full + s);
          } else {
            tma_load_2d(sa, &map_f, t.f0, t.row0 + d, full + s);
            tma_load_2d(sa + 8192, &map_f, t.f0 + 64, t.row0 + d, full + s);
          }
          for (int b = 0; b < boxes; ++b) {
            if (kMode == kGradW)
              tma_load_2d(sb + b * 8192, &map_t, t.c0 + 64 * b, t.row0 + d, full + s);
            else
              tma_load_2d(sb + b * kTokBox * 128, &map_t, d, t.row0 + kTokBox * b, full + s);
          }
        }
      }
      // before the block ends, its copies in flight land (bounded); after a
      // normal end warp 1 has waited for every one of them
      if (!ok) {
        for (uint32_t j = it > (uint32_t)kStages ? it - kStages : 0u; j < it; ++j)
          mbar_wait_bounded(full + j % kStages, (j / kStages) & 1u, kPolls);
      }
    }
  } else if (warp == 1) {
    uint32_t it = 0, done = 0;
    bool ok = true;
    for (int tile = first; ok && tile < tiles; tile += step) {
      const Tile t = tile_of<kMode, kTok>(a, table, tile);
      int c0, c1;
      share(t, c0, c1);
      if (c0 == c1) continue;
      const uint32_t buf = S::kSplit ? 0u : done & 1u;
      ok = __all_sync(0xffffffffu, wait_for(acc_empty + buf, ((S::kSplit ? done : done >> 1) & 1u) ^ 1u, gave_up));
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + buf * S::kAccCols;
      const int n = kMode == kGradW ? min(kTok, a.cols - t.c0) : t.n;
      const uint32_t idesc = instr_desc(a.bf16 != 0, kMode != kForward, kMode == kGradW, kFeat, (n + 15) & ~15);
      for (int c = c0; c < c1; ++c, ++it) {
        const uint32_t s = it % kStages, ph = (it / kStages) & 1u;
        ok = __all_sync(0xffffffffu, wait_for(full + s, ph, gave_up));
        if (!ok) break;
        unsigned char* sa = ring + s * S::kStage;
        unsigned char* sb = sa + S::kABytes;
        if (kMode == kGradW) {
          // lines of rows behind the expert's last one: zero in both operands
          // (whatever they held, NaN included, must not reach the sums)
          const int left = t.n - c * kDepth;
          if (left < kDepth) {
            const int lines = kDepth - left, blocks = 2 + (n + 63) / 64;
            for (int i = lane; i < blocks * lines * 8; i += 32) {
              const int line = i >> 3, blk = line / lines;
              *reinterpret_cast<uint4*>(sa + blk * 8192 + (left + line - blk * lines) * 128 + (i & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        tc_fence_after();
        if (lane == 0) {
          const uint32_t aa = smem_u32(sa), bb = smem_u32(sb);
          const uint64_t da = operand_desc(aa, kMode == kForward ? 16u : 8192u);
          const uint64_t db = operand_desc(bb, kMode == kGradW ? 8192u : 16u);
          constexpr uint32_t kStepA = (kMode == kForward ? 32 : 2048) >> 4, kStepB = (kMode == kGradW ? 2048 : 32) >> 4;
#pragma unroll
          for (uint32_t k = 0; k < kDepth / 16; ++k) {
            mma_f16(acc, da + k * kStepA, db + k * kStepB, idesc, c != c0 || k != 0);
            if (kGated)
              mma_f16(acc + kTok, operand_desc(aa + 16384u, 16u) + k * kStepA, db + k * kStepB, idesc,
                      c != c0 || k != 0);
          }
          mma_commit(empty + s);
          if (c + 1 == c1) mma_commit(acc_full + buf);
        }
        __syncwarp();
      }
      ++done;
    }
    if (!ok) {  // the products in flight end before their tensor memory is freed
      if (lane == 0) mma_commit(drained);
      __syncwarp();
      mbar_wait_bounded(drained, 0u, kPolls);
    }
  } else if (!S::kSplit) {
    const int quarter = warp & 3;  // the lanes of tensor memory this warp may read
    uint32_t done = 0;
    bool ok = true;
    for (int tile = first; tile < tiles; tile += step) {
      const Tile t = tile_of<kMode, kTok>(a, table, tile);
      const int f = t.f0 + quarter * 32 + lane;
      const bool mine = f < a.feat;
      const uint32_t buf = done & 1u;
      const bool sums = t.chunks > 0;
      if (sums) {
        ok = ok && __all_sync(0xffffffffu, wait_for(acc_full + buf, (done >> 1) & 1u, gave_up));
        tc_fence_after();
      }
      float b0 = 0.0f, b1 = 0.0f;
      if (kMode == kForward && a.bias && mine && t.expert < a.experts) {
        const int64_t at = (int64_t)t.expert * a.feat * (kGated ? 2 : 1) + f;
        b0 = load16(a.bias, at, a.bf16);
        if (kGated) b1 = load16(a.bias, at + a.feat, a.bf16);
      }
      const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16) + buf * S::kAccCols;
      const int n = kMode == kGradW ? min(kTok, a.cols - t.c0) : t.n;
      for (int c0 = 0; c0 < n; c0 += 32) {
        float v[32], up[kGated ? 32 : 1];
        if (sums && ok) {
          tmem_load32(acc + c0, v);
          if constexpr (kGated) tmem_load32(acc + kTok + c0, up);
          tmem_load_wait();
        } else {
          const float fill = ok ? 0.0f : __int_as_float(0x7fc00000);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            v[c] = fill;
            if constexpr (kGated) up[c] = fill;
          }
        }
        if (mine) {
          if constexpr (kMode == kGradW)
            store_row32(a, t, c0, f, v);
          else
            finish32<kGated>(a, t, c0, f, b0, b1, v, up, 0, 1);
        }
      }
      if (sums) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty + buf);
        ++done;
      }
    }
  }

  if constexpr (S::kSplit) {
    // one tile per cluster: the ranks' partials meet in shared memory
    __syncwarp();
    const bool busy = first < tiles;  // the same for all ranks of the cluster
    if (busy) {
      const Tile t = tile_of<kMode, kTok>(a, table, first);
      int s0, s1;
      share(t, s0, s1);
      const int quarter = warp & 3;
      const int f = t.f0 + quarter * 32 + lane;
      float v[32], up[kGated ? 32 : 1];
      float* red = reinterpret_cast<float*>(ring);  // [planes][kTok][kFeat]
      bool ok = true;
      if (warp >= 2) {
        if (s0 < s1) {
          ok = __all_sync(0xffffffffu, wait_for(acc_full, 0u, gave_up));
          tc_fence_after();
        }
        if (s0 < s1 && ok) {
          const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16);
          tmem_load32(acc, v);
          if constexpr (kGated) tmem_load32(acc + kTok, up);
          tmem_load_wait();
        } else {
          const float fill = ok ? 0.0f : __int_as_float(0x7fc00000);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            v[c] = fill;
            if constexpr (kGated) up[c] = fill;
          }
        }
        if (ranks > 1) {
          // every product has read its operands (acc_full), so the ring is free
          for (int c = 0; c < 32; ++c)
            if (c < t.n) {
              red[c * kFeat + quarter * 32 + lane] = v[c];
              if constexpr (kGated) red[(kTok + c) * kFeat + quarter * 32 + lane] = up[c];
            }
        }
      }
      if (ranks > 1) {
        __syncwarp();
        cluster_sync();
        if (warp >= 2) {
          // this rank finishes every ranks-th token
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            v[c] = 0.0f;
            if constexpr (kGated) up[c] = 0.0f;
            if (c < t.n && (c & (ranks - 1)) == rank) {
              for (int q = 0; q < ranks; ++q) {
                v[c] += cluster_load(smem_u32(red + c * kFeat + quarter * 32 + lane), q);
                if constexpr (kGated) up[c] += cluster_load(smem_u32(red + (kTok + c) * kFeat + quarter * 32 + lane), q);
              }
            }
          }
        }
      }
      if (warp >= 2 && f < a.feat) {
        float b0 = 0.0f, b1 = 0.0f;
        if (kMode == kForward && a.bias && t.expert < a.experts) {
          const int64_t at = (int64_t)t.expert * a.feat * (kGated ? 2 : 1) + f;
          b0 = load16(a.bias, at, a.bf16);
          if (kGated) b1 = load16(a.bias, at + a.feat, a.bf16);
        }
        finish32<kGated>(a, t, 0, f, b0, b1, v, up, rank, ranks);
      }
      if (ranks > 1) {
        __syncwarp();
        cluster_sync();  // no block leaves while another reads its partials
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_free(tmem, S::kTmemCols);
  if (threadIdx.x == 0 && *gave_up && a.status) atomicOr(a.status, LAPSUM_EXPERTS_TIMEOUT);
}

// ---- host -------------------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled g_encode = nullptr;

// a row-major [z][y][x] array of 16-bit values, rows `stride` values apart,
// copied in boxes of 64 x box_y x 1; positions outside read as zero
cudaError_t make_map(CUtensorMap* m, const void* base, int bf16, int64_t x, int64_t y, int64_t z, int64_t stride,
                     uint32_t box_y) {
  const cuuint64_t dims[3] = {(cuuint64_t)x, (cuuint64_t)y, (cuuint64_t)z};
  const cuuint64_t strides[2] = {(cuuint64_t)stride * 2, (cuuint64_t)stride * 2 * (cuuint64_t)y};
  const cuuint32_t box[3] = {64, box_y, 1}, unit[3] = {1, 1, 1};
  const CUresult r = g_encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                              z > 0 ? 3 : 2, const_cast<void*>(base), dims, strides, box, unit,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int kMode, int kTok, bool kGated>
cudaError_t allow_smem() {
  return cudaFuncSetAttribute(k_product<kMode, kTok, kGated>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Shape<kMode, kTok, kGated>::kSmem);
}

template <int kMode, int kTok, bool kGated>
cudaError_t launch(const char* name, const CUtensorMap& mf, const CUtensorMap& mt, const Args& a, int64_t grid,
                   int cluster, int tiles_grad_w, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Shape<kMode, kTok, kGated>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  Launch guard(name, st);
  return cudaLaunchKernelEx(&cfg, k_product<kMode, kTok, kGated>, mf, mt, a, tiles_grad_w);
}

// Forward and input gradient: the token side of a tile by the mean number of
// rows of an expert that can have any.
template <int kMode>
cudaError_t launch_rows(const char* name, const CUtensorMap& mf, const CUtensorMap& mt, const Args& a, bool gated,
                        int sms, cudaStream_t st) {
  const int64_t live = std::min<int64_t>(a.experts, a.rows);
  const int64_t mean = a.rows / std::max<int64_t>(1, live);
  const int64_t ftiles = (a.feat + kFeat - 1) / kFeat;
  // token tiles: at most one ragged one per expert (and one behind the last)
  auto bound = [&](int tok) { return (std::min<int64_t>(a.experts + 1, a.rows) + a.rows / tok) * ftiles; };
  if (mean <= 32) {
    const int64_t tiles = bound(32);
    const int chunks = (a.depth + kDepth - 1) / kDepth;
    int ranks = 1;
    while (ranks < 8 && tiles * ranks * 2 <= 2 * sms && chunks >= 8 * ranks) ranks *= 2;
    if constexpr (kMode == kForward)
      if (gated) return launch<kMode, 32, true>(name, mf, mt, a, tiles * ranks, ranks, 0, st);
    return launch<kMode, 32, false>(name, mf, mt, a, tiles * ranks, ranks, 0, st);
  }
  if constexpr (kMode == kForward)
    if (gated) return launch<kMode, 128, true>(name, mf, mt, a, std::min<int64_t>(bound(128), sms), 1, 0, st);
  if (mean <= 128) return launch<kMode, 128, false>(name, mf, mt, a, std::min<int64_t>(bound(128), sms), 1, 0, st);
  return launch<kMode, 256, false>(name, mf, mt, a, std::min<int64_t>(bound(256), sms), 1, 0, st);
}

Args base_args(const Product& p) {
  Args a{};
  a.rows = p.rows;
  a.experts = p.experts;
  a.bf16 = p.bf16;
  a.activation = p.activation;
  a.offsets = p.offsets;
  a.y = p.y;
  a.y_stride = p.y_stride;
  a.status = p.status;
  return a;
}

}  // namespace

cudaError_t linear_init() {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult got = cudaDriverEntryPointSymbolNotFound;
  cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &got);
  if (e != cudaSuccess) return e;
  if (!fn || got != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
  g_encode = reinterpret_cast<EncodeTiled>(fn);
  for (cudaError_t r : {allow_smem<kForward, 32, false>(), allow_smem<kForward, 32, true>(),
                        allow_smem<kForward, 128, false>(), allow_smem<kForward, 128, true>(),
                        allow_smem<kForward, 256, false>(), allow_smem<kGradX, 32, false>(),
                        allow_smem<kGradX, 128, false>(), allow_smem<kGradX, 256, false>(),
                        allow_smem<kGradW, 256, false>()})
    if (r != cudaSuccess) return r;
  return cudaSuccess;
}

cudaError_t launch_linear_fwd(const Product& p, int sms, cudaStream_t st) {
  const bool gated = p.activation == LAPSUM_ACT_SWIGLU;
  Args a = base_args(p);
  a.feat = (int)(gated ? p.out / 2 : p.out);
  a.depth = (int)p.in;
  a.bias = p.bias;
  a.residual = p.residual;
  a.residual_stride = p.residual_stride;
  a.preact = p.preact;
  a.preact_stride = p.preact_stride;
  CUtensorMap mf, mt;
  cudaError_t e = make_map(&mf, p.weight, p.bf16, p.in, p.out, p.experts, p.in, kFeat);
  if (e == cudaSuccess) e = make_map(&mt, p.x, p.bf16, p.in, p.rows, 0, p.x_stride, kTokBox);
  if (e != cudaSuccess) return e;
  return launch_rows<kForward>("k_product_fwd", mf, mt, a, gated, sms, st);
}

cudaError_t launch_linear_dx(const Product& p, int sms, cudaStream_t st) {
  Args a = base_args(p);
  a.feat = (int)p.in;
  a.depth = (int)p.out;
  CUtensorMap mf, mt;
  cudaError_t e = make_map(&mf, p.weight, p.bf16, p.in, p.out, p.experts, p.in, kDepth);
  if (e == cudaSuccess) e = make_map(&mt, p.grad_h, p.bf16, p.out, p.rows, 0, p.grad_h_stride, kTokBox);
  if (e != cudaSuccess) return e;
  return launch_rows<kGradX>("k_product_dx", mf, mt, a, false, sms, st);
}

cudaError_t launch_linear_dweight(const Product& p, int sms, cudaStream_t st) {
  Args a = base_args(p);
  a.feat = (int)p.out;
  a.cols = (int)p.in;
  CUtensorMap mf, mt;
  cudaError_t e = make_map(&mf, p.grad_h, p.bf16, p.out, p.rows, 0, p.grad_h_stride, kDepth);
  if (e == cudaSuccess) e = make_map(&mt, p.x, p.bf16, p.in, p.rows, 0, p.x_stride, kDepth);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)p.experts * ((p.out + kFeat - 1) / kFeat) * ((p.in + 255) / 256);
  return launch<kGradW, 256, false>("k_product_dw", mf, mt, a, std::min<int64_t>(tiles, sms), 1, (int)tiles, st);
}

}  // namespace lapsum
