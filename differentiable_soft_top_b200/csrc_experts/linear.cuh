// linear.cuh -- the experts' products and their gradients on the tensor cores.
//
// y_r = act(W_e x_r + b_e) + residual_r for the rows of expert e.  Rows are
// few or many per expert and start anywhere, the features of a weight matrix
// are many and regular; so the weights take the fixed side of the matrix
// instruction (M = 128 of its rows) and the tokens the variable one (N = 16 ..
// 256): D^T = W X^T.  A tile with 5 tokens then costs an N = 16 instruction,
// not a 128-row one, and one kernel serves one token and long prompts.
//
//   forward          D[f, t] = sum_k W[f, k] X[t, k]       both K major
//   input gradient   D[k, t] = sum_n W[n, k] dH[t, n]      W MN major
//   weight gradient  D[n, k] = sum_t dH[t, n] X[t, k]      both MN major; the
//                    contraction runs over an expert's rows and its ragged
//                    end is zeroed in shared memory
//
// In a block warp 0 fills a ring of stages by tiled copies (64 deep, 128-byte
// swizzle), warp 1 issues the products, the other four or eight read the
// accumulators from tensor memory and write the result.  (For weight gradients
// one more warp zeroes the ragged ends.)  Two accumulators let
// the epilogue of one tile run beside the products of the next; blocks walk
// the tiles with a stride of the grid.  Three forms, by the rows of an expert:
//   many   two blocks work as a pair on 256 features x 256 tokens: each copies
//          its 128 features and half of the tokens, 32 KB per 64 of depth
//          where a block alone would copy 48 KB, more than L2 delivers in the
//          512 cycles of that product
//   some   one block, 128 tokens
//   few    one block, 32 tokens, two blocks per SM; where there are fewer tiles
//          than that, one tile per cluster of 2, 4 or 8 blocks, which split the
//          contraction and join their fp32 partials through distributed shared
//          memory in the order of rank
//
// Gated weights (silu(gate) * up) are copied interleaved, 8 rows of one and 8
// of the other, so that a thread holds the gate and the up value of a feature.
// The epilogue reads accumulators as 8 x 8 fragments, which the transposing
// stores turn into rows of the output in shared memory: global accesses are 16
// bytes per lane.
//
// Every wait is bounded: a block that gives up sets a status bit, writes NaN
// for what it leaves undone, lets its copies land and frees its tensor memory.
#pragma once

#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "activation.cuh"
#include "chain.cuh"
#include "experts.h"
#include "umma.cuh"

namespace lapsum {
namespace {

enum Mode { kForward, kGradX, kGradW };

constexpr int kDepth = 64;              // contraction per stage: one 128-byte line
constexpr int kLanes = 128;             // accumulator lanes of a block
constexpr int kTokBox = 32;             // tokens per copied box of a ragged tile (a full one: one box)
constexpr int kGroup = 16;              // token tiles that share their features' tiles in time
constexpr int kPitch = 80;              // bytes between staged rows of 64: conflict-free

struct Args {
  int64_t rows;
  int experts, activation;
  int feat;          // features of the output (half of the weights' rows when gated)
  int depth;         // contraction length (kGradW: set per tile)
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
  uint32_t polls;    // of a bounded wait before it gives up
  int starve;        // test knob: nothing is copied, so that waits run out
};

template <int kMode, int kTok, bool kGated, bool kSplit>
struct Shape {
  static constexpr bool kPair = kTok == 256;
  static constexpr bool kFew = kTok == 32;         // two blocks per SM
  static constexpr int kEpilogue = kFew ? 4 : 8;    // warps: one or two per quarter of the lanes
  static constexpr int kThreads = 64 + 32 * kEpilogue + (kMode == kGradW ? 32 : 0);
  static constexpr int kFeat = kLanes / (kGated ? 2 : 1);           // features of a block's tile
  static constexpr int kTileFeat = kFeat * (kPair ? 2 : 1);         // of a tile
  static constexpr int kABytes = kLanes * 128;
  static constexpr int kBBytes = (kPair ? kTok / 2 : kTok) * 128;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kStages = kFew ? 4 : 196 * 1024 / kStage;
  static constexpr int kTmemCols = kSplit ? 32 : 2 * kTok;
  // (the split form stages in the ring; here its ranks' partials arrive)
  static constexpr int kStaging = kSplit ? 32 * kLanes * 4 : kEpilogue * 32 * kPitch;
  static constexpr int kTable = kMode == kGradW ? 0 : (LAPSUM_EXPERTS_MAX + 2) * 4;
  static constexpr int kSmem = kStages * kStage + kStaging + kTable + 1024 /* alignment */ + 512 /* barriers */;
};

// ---- 16-bit values ------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  return unpack2<T>((uint32_t)__ldg(static_cast<const uint16_t*>(p) + i)).x;
}

// ---- tiles ------------------------------------------------------------------------------
struct Tile {
  int expert;
  int row0, n;   // tokens [row0, row0 + n) (kGradW: the expert's rows)
  int f0;        // first feature of this block
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
// experts + 1.  The whole block; ends with the block in step.
template <int kTok>
__device__ __forceinline__ void build_table(const Args& a, int* table) {
  const int lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e <= a.experts; e += blockDim.x) {
    int lo, n;
    row_range(a, e, lo, n);
    table[e] = (n + kTok - 1) / kTok;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int base = 0;
    for (int e0 = 0; e0 <= a.experts; e0 += 32) {
      const int e = e0 + lane, own = e <= a.experts ? table[e] : 0;
      int v = own;
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
  __syncthreads();
}

template <int kMode, int kTok, bool kGated, bool kSplit>
__device__ __forceinline__ Tile tile_of(const Args& a, const int* table, int tile, int half) {
  using S = Shape<kMode, kTok, kGated, kSplit>;
  Tile t;
  const int ftiles = (a.feat + S::kTileFeat - 1) / S::kTileFeat;
  t.c0 = 0;
  if (kMode == kGradW) {
    const int ctiles = (a.cols + kTok - 1) / kTok;
    t.expert = tile / (ftiles * ctiles);
    const int in = tile - t.expert * (ftiles * ctiles);
    t.f0 = (in / ctiles) * S::kTileFeat + half * S::kFeat;
    t.c0 = (in % ctiles) * kTok;
    row_range(a, t.expert, t.row0, t.n);
    t.chunks = (t.n + kDepth - 1) / kDepth;
    return t;
  }
  int lo = 0, hi = a.experts;  // the last expert whose first tile is <= tt
  const int tt = tile / ftiles;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (table[mid] <= tt) lo = mid; else hi = mid - 1;
  }
  t.expert = lo;
  int row0, n;
  row_range(a, lo, row0, n);
  // An expert's tiles go in groups of up to kGroup token tiles, each feature
  // tile of the group's next to one another: what runs at one time then reads
  // about as many rows of the weights as of the tokens, not all of the weights.
  const int in = tile - table[lo] * ftiles, count = table[lo + 1] - table[lo];
  const int group = in / (kGroup * ftiles), wide = min(kGroup, count - group * kGroup);
  const int rest = in - group * kGroup * ftiles, f = rest / wide;
  t.f0 = f * S::kTileFeat + half * S::kFeat;
  // Its rows are spread evenly over its tiles (in steps of 32, the last one gets
  // the rest): every block's tiles cost about the same, where full tiles and a
  // small one last left some blocks with more work (32768 rows over 64 experts
  // of 256 to 768: 431 us, 313 us with 512 each).
  const int share = ((n + count - 1) / count + 31) & ~31;
  const int skip = (group * kGroup + rest - f * wide) * share;
  t.row0 = row0 + skip;
  t.n = min(n - skip, share);
  t.chunks = lo < a.experts ? (a.depth + kDepth - 1) / kDepth : 0;
  return t;
}

// ---- bounded waits: a block that has given up somewhere gives up everywhere --------------
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile uint32_t* gave_up, uint32_t polls) {
  for (uint32_t i = 0; i < polls; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 63u && *gave_up) return false;
  }
  *gave_up = 1u;
  return false;
}
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile uint32_t* gave_up, uint32_t polls) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, gave_up, polls);
}

// ---- epilogue: a warp's 32 accumulator lanes x 32 columns --------------------------------
// v[h]: the fragments of lanes 16 h .. 16 h + 15 (tmem_load_16x32).  Without
// gates lane = feature; with gates lanes 16 h + 0..7 are the gates and + 8..15 the
// ups of features 8 h .. 8 h + 7.  p[j]: packed pairs of tokens 8 j + c, + 1 of the
// feature groups (of 8) in order: 4 (2 with gates) per token group j.
template <bool kGated>
struct Frag {
  static constexpr int kGroups = kGated ? 2 : 4;
  uint32_t p[4][kGroups];
};

// bytes from the staging area: token `tok`, feature group `g`
__device__ __forceinline__ uint32_t staged(uint32_t base, int tok, int g) { return base + tok * kPitch + g * 16; }

template <bool kGated>
__device__ __forceinline__ uint32_t lane_row(uint32_t base, int jj, int lane) {
  const int m = lane >> 3;
  return kGated ? staged(base, 8 * (jj + (m >> 1)) + (lane & 7), m & 1) : staged(base, 8 * jj + (lane & 7), m);
}

// fragments -> rows of dst (16 bytes per lane).  own: which (token group j,
// lane half h) pieces are this block's to write, bit 2 j + h.
template <bool kGated>
__device__ __forceinline__ void put(const Frag<kGated>& f, uint32_t base, void* dst, int64_t row, int64_t stride, int feat0,
                                    int feat, int n, uint32_t own, int lane) {
  constexpr int G = Frag<kGated>::kGroups;
  if (kGated) {
#pragma unroll
    for (int j = 0; j < 4; j += 2)
      stage_4<true>(lane_row<kGated>(base, j, lane), f.p[j][0], f.p[j][1], f.p[j + 1][0], f.p[j + 1][1]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      stage_4<true>(lane_row<kGated>(base, j, lane), f.p[j][0], f.p[j][1], f.p[j][2 % G], f.p[j][3 % G]);
  }
  __syncwarp();
  uint16_t* out = static_cast<uint16_t*>(dst);
#pragma unroll
  for (int it = 0; it < G; ++it) {
    const int tok = it * (32 / G) + lane / G, g = lane % G;
    const int h = kGated ? g : g >> 1;
    const uint4 v = lds16(staged(base, tok, g));
    if (tok < n && feat0 + 8 * g < feat && (own >> (2 * (tok >> 3) + h) & 1u))
      *reinterpret_cast<uint4*>(out + (row + tok) * stride + feat0 + 8 * g) = v;
  }
  __syncwarp();
}

// rows of src, one chunk: loads only
template <bool kGated>
__device__ __forceinline__ void get_rows(uint4 (&q)[Frag<kGated>::kGroups], const void* src, int64_t row, int64_t stride,
                                         int feat0, int feat, int n, int lane) {
  constexpr int G = Frag<kGated>::kGroups;
  const uint16_t* in = static_cast<const uint16_t*>(src);
#pragma unroll
  for (int it = 0; it < G; ++it) {
    const int tok = it * (32 / G) + lane / G, g = lane % G;
    q[it] = make_uint4(0u, 0u, 0u, 0u);
    if (tok < n && feat0 + 8 * g < feat)
      q[it] = __ldg(reinterpret_cast<const uint4*>(in + (row + tok) * stride + feat0 + 8 * g));
  }
}

// 32 tokens of a warp's features: bias, activation, residual, store
template <typename T, bool kGated>
__device__ __forceinline__ void finish(const Args& a, const Tile& t, int c0, int feat0, const float (&bias)[4],
                                       float (&v)[2][16], const uint4 (&res)[Frag<kGated>::kGroups], uint32_t base,
                                       uint32_t own, int lane) {
  constexpr int G = Frag<kGated>::kGroups;
  const int n = min(32, t.n - c0);
  const int64_t row = t.row0 + c0;
  const bool multiplied = t.expert < a.experts;
  Frag<kGated> f;
  float o[4][G][2];
  if (multiplied) {
    if (a.bias) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 16; ++i) v[h][i] += bias[2 * h + (i >> 1 & 1)];
    }
    if (a.preact) {
      // What fp16 cannot hold as it is: what relu passes stays positive (the type
      // ends at 2^-24, and its gradient asks for the sign), and what is finite stays
      // finite (y often is where h is not, as silu of -7e4, and an infinity would turn
      // a gradient that vanishes into NaN).  In what is kept only: y does not change.
      bool odd = false;
      if constexpr (std::is_same<T, __half>::value) {
        float big = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) big = fmaxf(big, fmaxf(fabsf(v[0][i]), fabsf(v[1][i])));
        odd = __any_sync(0xffffffffu, big > 65504.0f) || (!kGated && a.activation == LAPSUM_ACT_RELU);
      }
      auto kept = [&](float x) {
        if (!kGated && a.activation == LAPSUM_ACT_RELU && x > 0.0f) x = fmaxf(x, 6e-8f);
        return fabsf(x) > 65504.0f && fabsf(x) < INFINITY ? copysignf(65504.0f, x) : x;
      };
#pragma unroll
      for (int up = 0; up < (kGated ? 2 : 1); ++up) {
        // gated: lane half g's gates or ups; else group g
        auto pair = [&](int j, int g, auto as) {
          const float(&from)[16] = v[kGated ? g : g >> 1];
          const int at = 4 * j + 2 * (kGated ? up : g & 1);
          f.p[j][g] = pack2<T>(as(from[at]), as(from[at + 1]));
        };
        if (odd) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int g = 0; g < G; ++g) pair(j, g, kept);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int g = 0; g < G; ++g) pair(j, g, [](float x) { return x; });
        }
        put<kGated>(f, base, static_cast<uint16_t*>(a.preact) + up * a.feat, row, a.preact_stride, feat0, a.feat, n, own,
                    lane);
      }
    }
    if (kGated) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float g = v[h][4 * j + i];
            o[j][h][i] = g * sigmoid_of(g) * v[h][4 * j + 2 + i];
          }
    } else {
      activate(v[0], a.activation);
      activate(v[1], a.activation);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int i = 0; i < 2; ++i) o[j][g][i] = v[g >> 1][4 * j + 2 * (g & 1) + i];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int g = 0; g < G; ++g) o[j][g][0] = o[j][g][1] = 0.0f;
  }
  if (a.residual) {  // rows -> fragments
#pragma unroll
    for (int it = 0; it < G; ++it) sts16(staged(base, it * (32 / G) + lane / G, lane % G), res[it]);
    __syncwarp();
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; j += kGated ? 2 : 1) {
      fetch_4_trans(lane_row<kGated>(base, j, lane), r[0], r[1], r[2], r[3]);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float2 w = unpack2<T>(r[m]);
        float* to = kGated ? o[j + (m >> 1)][m & 1] : o[j][m % G];
        to[0] += w.x;
        to[1] += w.y;
      }
    }
    __syncwarp();
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int g = 0; g < G; ++g) f.p[j][g] = pack2<T>(o[j][g][0], o[j][g][1]);
  put<kGated>(f, base, a.y, row, a.y_stride, feat0, a.feat, n, own, lane);
}

// 32 columns of a warp's 32 rows of a weight gradient
template <typename T>
__device__ __forceinline__ void finish_grad_w(const Args& a, const Tile& t, int c0, int feat0, const float (&v)[2][16],
                                              uint32_t base, int lane) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int r = 0; r < 2; ++r)  // 8 rows, four groups of 8 columns
      stage_4<false>(staged(base, 16 * h + 8 * r + (lane & 7), lane >> 3), pack2<T>(v[h][2 * r], v[h][2 * r + 1]),
                     pack2<T>(v[h][4 + 2 * r], v[h][5 + 2 * r]), pack2<T>(v[h][8 + 2 * r], v[h][9 + 2 * r]),
                     pack2<T>(v[h][12 + 2 * r], v[h][13 + 2 * r]));
  __syncwarp();
  uint16_t* out = static_cast<uint16_t*>(a.y);
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int r = it * 8 + lane / 4, col = t.c0 + c0 + 8 * (lane & 3);
    const uint4 w = lds16(staged(base, r, lane & 3));
    if (feat0 + r < a.feat && col < a.cols)
      *reinterpret_cast<uint4*>(out + ((int64_t)t.expert * a.feat + feat0 + r) * a.cols + col) = w;
  }
  __syncwarp();
}

template <typename T, bool kGated>
__device__ __forceinline__ void load_bias(const Args& a, const Tile& t, int feat0, float (&b)[4], int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = 0.0f;
  if (!a.bias || t.expert >= a.experts) return;
  const int64_t at = (int64_t)t.expert * a.feat * (kGated ? 2 : 1);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int f = feat0 + (kGated ? 8 * (i >> 1) : 8 * i) + lane / 4;
    if (f < a.feat) b[i] = load1<T>(a.bias, at + f + (kGated && (i & 1) ? a.feat : 0));
  }
}

__device__ __forceinline__ void fill(float (&v)[2][16], float x) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[0][i] = v[1][i] = x;
}

// map_f: the weights (kGradW: dH); map_t: the tokens' rows in small boxes,
// map_full: in boxes of a full tile
template <typename T, int kMode, int kTok, bool kGated, bool kSplit>
__global__ void __launch_bounds__(Shape<kMode, kTok, kGated, kSplit>::kThreads, kTok == 32 ? 2 : 1)
    k_product(const __grid_constant__ CUtensorMap map_f, const __grid_constant__ CUtensorMap map_t,
              const __grid_constant__ CUtensorMap map_full, const Args a, int tiles_grad_w) {
  using S = Shape<kMode, kTok, kGated, kSplit>;
  constexpr int kStages = S::kStages;
  constexpr bool kPair = S::kPair;
  extern __shared__ unsigned char smem_raw[];
  // operands in the 128-byte swizzle start on 1024-byte boundaries
  unsigned char* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char* staging = ring + kStages * S::kStage;
  unsigned char* tail = staging + S::kStaging;
  uint64_t* full = reinterpret_cast<uint64_t*>(tail);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;      // [2]
  uint64_t* acc_empty = acc_full + 2;        // [2]
  uint64_t* drained = acc_empty + 2;
  uint64_t* landed = drained + 1;            // kGradW [kStages]: copies of a ragged end
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(landed + kStages);
  volatile uint32_t* gave_up = tmem_at + 1;
  int* table = reinterpret_cast<int*>(tail + 512);

  if (kSplit) cluster_arrive();  // waited for before the first access to another block's memory
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = kPair ? (int)cluster_rank() : 0;
  if (threadIdx.x == 0) {
    prefetch_map(&map_f);
    prefetch_map(&map_t);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, kPair ? 2 : 1);  // kPair: of the first block, for both blocks' copies
      mbar_init(empty + s, 1);
      mbar_init(landed + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + b, 1);
      mbar_init(acc_empty + b, S::kEpilogue * (kPair ? 2 : 1));
    }
    mbar_init(drained, 1);
    *gave_up = 0u;
  }
  if (warp == 1) {
    tmem_alloc<kPair>(tmem_at, S::kTmemCols);
    // Not before: the next kernel may take tensor memory too, and this block's must
    // not come behind that of a kernel which waits for this one's end.
    grid_launch_next();
  }
  grid_wait_previous();  // from here on the kernels before this one have finished
  if (kMode != kGradW) build_table<kTok>(a, table);
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();  // the other block's barriers are set up
  tc_fence_after();
  const uint32_t tmem = *tmem_at;

  const int ftiles = (a.feat + S::kTileFeat - 1) / S::kTileFeat;
  const int tiles = kMode == kGradW ? tiles_grad_w : table[a.experts + 1] * ftiles;
  const int ranks = kSplit ? (int)cluster_size() : kPair ? 2 : 1;
  const int rank = kSplit ? (int)cluster_rank() : 0;
  // few rows: the grid holds a cluster for every tile there can be
  const int first = (int)blockIdx.x / ranks, step = kSplit ? max(tiles, 1) : (int)gridDim.x / ranks;

  // kSplit: this block's share of a tile's contraction
  auto share = [&](const Tile& t, int& c0, int& c1) {
    if (!kSplit) {
      c0 = 0;
      c1 = t.chunks;
      return;
    }
    const int per = (t.chunks + ranks - 1) / ranks;
    c0 = min(rank * per, t.chunks);
    c1 = min(c0 + per, t.chunks);
  };
  // variable side of the instruction, and the part of it this block copies
  auto width = [&](const Tile& t, int& n, int& n0, int& own) {
    const int all = kMode == kGradW ? min(kTok, a.cols - t.c0) : t.n;
    n = kPair ? (all + 31) & ~31 : (all + 15) & ~15;
    n0 = half * (n / 2);
    own = kPair ? min(n / 2, max(all - n0, 0)) : all;
  };

  if (warp == 0) {
    if (lane == 0) {
      uint32_t s = 0, ph = 0, used = 0;  // stage, its phase, stages filled (at most kStages)
      uint32_t ends = 0, phases = 0;     // kGradW, a bit per stage: holds a ragged end; its barrier's phase
      bool ok = true;
      for (int tile = first; ok && tile < tiles; tile += step) {
        const Tile t = tile_of<kMode, kTok, kGated, kSplit>(a, table, tile, half);
        int c0, c1, n, n0, own;
        share(t, c0, c1);
        width(t, n, n0, own);
        constexpr int kBox = kMode == kGradW ? 64 : kTokBox, kBoxBytes = kMode == kGradW ? 8192 : kTokBox * 128;
        // more than two small boxes: one of the full height (rows beyond the tile's
        // are copied in vain; what limits is the number of copies)
        const bool whole = kMode != kGradW && !S::kFew && own > 2 * kTokBox;
        const int boxes = (own + kBox - 1) / kBox;
        const uint32_t bytes = S::kABytes + (whole ? S::kBBytes : boxes * kBoxBytes);
        for (int c = c0; c < c1; ++c) {
          if (a.starve || !wait_for(empty + s, ph ^ 1u, gave_up, a.polls)) {
            ok = false;
            break;
          }
          unsigned char* sa = ring + s * S::kStage;
          unsigned char* sb = sa + S::kABytes;
          const int d = c * kDepth;
          // a ragged end is full when the zeroing warp says so
          const bool end = kMode == kGradW && t.n - d < kDepth;
          if (kMode == kGradW) {
            ends = end ? ends | 1u << s : ends & ~(1u << s);
            if (end) phases ^= 1u << s;
          }
          const uint32_t bar = end ? smem_u32(landed + s) : kPair ? in_block(full + s, 0) : smem_u32(full + s);
          if (kPair && !end)
            arrive_expect_at(bar, bytes);
          else
            mbar_arrive_expect_tx(end ? landed + s : full + s, bytes);
          if (kMode == kForward) {
            if (kGated)
              tma_load_5d<kPair>(sa, &map_f, d, 0, 0, t.f0 / 8, t.expert, bar);
            else
              tma_load_3d<kPair>(sa, &map_f, d, t.f0, t.expert, bar);
          } else if (kMode == kGradX) {
            tma_load_3d<kPair>(sa, &map_f, t.f0, d, t.expert, bar);
            tma_load_3d<kPair>(sa + 8192, &map_f, t.f0 + 64, d, t.expert, bar);
          } else {
            tma_load_2d<kPair>(sa, &map_f, t.f0, t.row0 + d, bar);
            tma_load_2d<kPair>(sa + 8192, &map_f, t.f0 + 64, t.row0 + d, bar);
          }
          if (whole) tma_load_2d<kPair>(sb, &map_full, d, t.row0 + n0, bar);
          for (int b = whole ? boxes : 0; b < boxes; ++b) {
            if (kMode == kGradW)
              tma_load_2d<kPair>(sb + b * kBoxBytes, &map_t, t.c0 + n0 + kBox * b, t.row0 + d, bar);
            else
              tma_load_2d<kPair>(sb + b * kBoxBytes, &map_t, d, t.row0 + n0 + kBox * b, bar);
          }
          if (used < kStages) ++used;
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // Before the block ends, its copies in flight land (bounded); after a normal
      // end warp 1 of this block, or of the pair's first, has waited for every one
      // of them.  In a pair that ends early the first block looks after both: it
      // arrives in place of what it would have copied to the stages that the
      // second may have filled ahead of it, and waits for all stages.
      if (!ok && (!kPair || half == 0)) {
        const uint32_t s1 = s, ph1 = ph;
        for (; used; --used) {
          if (s == 0) ph ^= 1u;
          s = s == 0 ? kStages - 1 : s - 1;
          if (kMode == kGradW && (ends >> s & 1u))
            mbar_wait_bounded(landed + s, (phases >> s & 1u) ^ 1u, a.polls);
          else
            mbar_wait_bounded(full + s, ph, a.polls);
        }
        s = s1, ph = ph1;
        for (int i = 0; kPair && i < kStages; ++i) {
          mbar_arrive(full + s);
          mbar_wait_bounded(full + s, ph, a.polls);
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    }
  } else if (warp == 1) {
    // One lane issues, in a pair that of the first block.
    if (lane == 0 && half == 0) {
      uint32_t s = 0, ph = 0, done = 0;
      bool ok = true;
      int tile = first;
      Tile t = tile_of<kMode, kTok, kGated, kSplit>(a, table, min(tile, max(tiles - 1, 0)), half);
      for (; ok && tile < tiles; tile += step) {
        const Tile cur = t;
        int c0, c1, n, n0, own;
        share(cur, c0, c1);
        width(cur, n, n0, own);
        if (c0 < c1) {
          const uint32_t buf = kSplit ? 0u : done & 1u;
          ok = wait_for(acc_empty + buf, ((kSplit ? done : done >> 1) & 1u) ^ 1u, gave_up, a.polls);
          tc_fence_after();
          const uint32_t acc = tmem + buf * kTok;
          const uint32_t idesc = instr_desc(std::is_same<T, __nv_bfloat16>::value, kMode != kForward, kMode == kGradW,
                                            kLanes * (kPair ? 2 : 1), n);
          for (int c = c0; ok && c < c1; ++c) {
            ok = wait_for(full + s, ph, gave_up, a.polls);
            if (!ok) break;
            const int left = kMode == kGradW ? cur.n - c * kDepth : kDepth;
            if (kPair && left < kDepth) mbar_try_wait_cluster(full + s, ph);  // done already: acquires the zeroed lines
            tc_fence_after();
            const uint32_t sa = smem_u32(ring) + s * S::kStage;
            const uint64_t da = operand_desc(sa, kMode == kForward ? 16u : 8192u);
            const uint64_t db = operand_desc(sa + S::kABytes, kMode == kGradW ? 8192u : 16u);
            constexpr uint32_t kStepA = (kMode == kForward ? 32 : 2048) >> 4,
                               kStepB = (kMode == kGradW ? 2048 : 32) >> 4;
#pragma unroll
            for (uint32_t k = 0; k < kDepth / 16; ++k)
              if (kMode != kGradW || (int)(16 * k) < left)
                mma_f16<kPair>(acc, da + k * kStepA, db + k * kStepB, idesc, c != c0 || k != 0);
            mma_commit<kPair>(empty + s);
            if (c + 1 == c1) mma_commit<kPair>(acc_full + buf);
            if (++s == kStages) {
              s = 0;
              ph ^= 1u;
            }
          }
          ++done;
        }
        // the next tile is found while this one's products run
        if (tile < tiles - step) t = tile_of<kMode, kTok, kGated, kSplit>(a, table, tile + step, half);
      }
      if (!ok) {  // the products in flight end before their tensor memory is freed
        mma_commit<kPair>(drained);
        mbar_wait_bounded(drained, 0u, a.polls);
      }
    }
  } else if (kMode == kGradW && warp == 2 + S::kEpilogue) {
    // The products take whole steps of 16 rows: in the last step of an expert
    // the lines behind its rows are zeroed in both operands (whatever they held,
    // NaN included, must not reach the sums).  A lane has 16 bytes of one of the
    // four blocks of 64 columns.
    uint32_t next = 0, phases = 0;  // the tile's first stage; a parity per stage
    bool ok = true;
    for (int tile = first; ok && tile < tiles; tile += step) {
      const Tile t = tile_of<kMode, kTok, kGated, kSplit>(a, table, tile, half);
      next += t.chunks;
      const int left = t.n & (kDepth - 1);
      if (left == 0) continue;
      int n, n0, own;
      width(t, n, n0, own);
      const uint32_t s = (next - 1) % kStages;
      ok = __all_sync(0xffffffffu, wait_for(landed + s, phases >> s & 1u, gave_up, a.polls));
      phases ^= 1u << s;
      if (!ok) break;
      if ((lane >> 3) < 2 + (own + 63) / 64) {
        const uint32_t to = smem_u32(ring) + s * S::kStage + (lane >> 3) * 8192 + (lane & 7) * 16;
        for (int line = left; line & 15; ++line) sts16(to + line * 128, make_uint4(0u, 0u, 0u, 0u));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_at<true>(in_block(full + s, 0));
    }
  } else if (!kSplit) {
    // Two warps share a quarter of the lanes and take every other 32 columns.
    const int quarter = warp & 3, part = (warp - 2) >> 2;
    const uint32_t base = smem_u32(staging) + (warp - 2) * 32 * kPitch;
    uint32_t done = 0;
    bool ok = true;
    for (int tile = first; tile < tiles; tile += step) {
      const Tile t = tile_of<kMode, kTok, kGated, kSplit>(a, table, tile, half);
      const int feat0 = t.f0 + quarter * (S::kFeat / 4);
      const uint32_t buf = done & 1u;
      const bool sums = t.chunks > 0;
      const int n = kMode == kGradW ? min(kTok, a.cols - t.c0) : t.n;
      float bias[4];
      uint4 res[Frag<kGated>::kGroups];
      if (kMode == kForward) {
        load_bias<T, kGated>(a, t, feat0, bias, lane);
        if (a.residual && 32 * part < n)
          get_rows<kGated>(res, a.residual, t.row0 + 32 * part, a.residual_stride, feat0, a.feat, n - 32 * part, lane);
      }
      if (sums) {
        ok = ok && __all_sync(0xffffffffu, wait_for(acc_full + buf, (done >> 1) & 1u, gave_up, a.polls));
        tc_fence_after();
      }
      auto release = [&] {  // this warp's columns are in registers
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (kPair) arrive_at<false>(in_block(acc_empty + buf, 0));
          else mbar_arrive(acc_empty + buf);
        }
      };
      const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16) + buf * kTok;
      if (sums && ok && 32 * part >= n) release();
      for (int c0 = 32 * part; c0 < n; c0 += 64) {
        float v[2][16];
        if (sums && ok) {
          tmem_load_16x32(acc + c0, v[0]);
          tmem_load_16x32(acc + (16u << 16) + c0, v[1]);
          tmem_load_wait();
          if (c0 + 64 >= n) release();
        } else {
          fill(v, ok ? 0.0f : __int_as_float(0x7fc00000));
        }
        if constexpr (kMode == kGradW) {
          finish_grad_w<T>(a, t, c0, feat0, v, base, lane);
        } else {
          uint4 cur[Frag<kGated>::kGroups];
#pragma unroll
          for (int i = 0; i < Frag<kGated>::kGroups; ++i) cur[i] = res[i];
          if (kMode == kForward && a.residual && c0 + 64 < n)  // the next chunk's, while this one is worked on
            get_rows<kGated>(res, a.residual, t.row0 + c0 + 64, a.residual_stride, feat0, a.feat, n - c0 - 64, lane);
          finish<T, kGated>(a, t, c0, feat0, bias, v, cur, base, 0xffu, lane);
        }
      }
      if (sums) ++done;
    }
  }

  if constexpr (kSplit) {
    // one tile per cluster: the ranks' partials meet in shared memory
    __syncwarp();
    cluster_wait();  // every block has started
    const bool busy = first < tiles;  // the same for all ranks of the cluster
    if (busy) {
      const Tile t = tile_of<kMode, kTok, kGated, kSplit>(a, table, first, 0);
      int s0, s1;
      share(t, s0, s1);
      const int quarter = warp & 3;
      const int feat0 = t.f0 + quarter * (S::kFeat / 4);
      float v[2][16], bias[4];
      uint4 res[Frag<kGated>::kGroups];
      // every product has read its operands (acc_full), so the ring is free
      const uint32_t base = smem_u32(ring) + quarter * 32 * kPitch;
      // A piece is 8 tokens x 16 lanes (4 values of a thread), piece p the one of
      // tokens 8 (p / 2) .. and lanes 16 (p % 2) ..; rank p % ranks joins it.
      // partials[rank][value][thread], 32 values in all: each rank sends the
      // pieces of the others to where they are joined.
      const uint32_t partials = smem_u32(staging) + ((quarter << 5) + lane) * 4;
      const int each = 32 / ranks;
      bool ok = true;
      if (warp >= 2) {
        load_bias<T, kGated>(a, t, feat0, bias, lane);
        if (a.residual) get_rows<kGated>(res, a.residual, t.row0, a.residual_stride, feat0, a.feat, t.n, lane);
        if (s0 < s1) {
          ok = __all_sync(0xffffffffu, wait_for(acc_full, 0u, gave_up, a.polls));
          tc_fence_after();
        }
        if (s0 < s1 && ok) {
          const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16);
          tmem_load_16x32(acc, v[0]);
          tmem_load_16x32(acc + (16u << 16), v[1]);
          tmem_load_wait();
        } else {
          fill(v, ok ? 0.0f : __int_as_float(0x7fc00000));
        }
        if (ranks > 1) {
#pragma unroll
          for (int p = 0; p < 8; ++p)
            if (8 * (p >> 1) < t.n) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                cluster_store(partials + (rank * each + p / ranks * 4 + i) * (kLanes * 4), p & (ranks - 1),
                              v[p & 1][4 * (p >> 1) + i]);
            }
        }
      }
      uint32_t own = 0xffu;
      if (ranks > 1) {
        __syncwarp();
        cluster_sync();  // nothing goes between the blocks after this
        own = ranks == 8 ? 1u << rank : ranks == 4 ? 0x11u << rank : 0x55u << rank;
        if (warp >= 2) {
#pragma unroll
          for (int p = 0; p < 8; ++p)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float sum = 0.0f;
              if (8 * (p >> 1) < t.n && (own >> p & 1u))
                for (int q = 0; q < ranks; ++q) sum += lds4(partials + (q * each + p / ranks * 4 + i) * (kLanes * 4));
              v[p & 1][4 * (p >> 1) + i] = sum;
            }
        }
      }
      if (warp >= 2) finish<T, kGated>(a, t, 0, feat0, bias, v, res, base, own, lane);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();  // no block leaves while the pair's products or arrivals are under way
  tc_fence_after();
  if (warp == 1) tmem_free<kPair>(tmem, S::kTmemCols);
  if (threadIdx.x == 0 && *gave_up && a.status) atomicOr(a.status, LAPSUM_EXPERTS_TIMEOUT);
}

// ---- host -------------------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled g_encode = nullptr;

// Tensor maps of 16-bit arrays, copied in boxes with 64 values along x in the
// 128-byte swizzle; positions outside read as zero.  The swizzle does not look
// at the type, so both 16-bit types are copied as bf16.
cudaError_t encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                   const cuuint32_t* box) {
  const cuuint32_t unit[5] = {1, 1, 1, 1, 1};
  const CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, unit,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
cudaError_t map_rows(CUtensorMap* m, const void* base, int64_t x, int64_t rows, int64_t stride, uint32_t box_y) {
  const cuuint64_t dims[2] = {(cuuint64_t)x, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t box[2] = {64, box_y};
  return encode(m, base, 2, dims, strides, box);
}
cudaError_t map_weights(CUtensorMap* m, const void* base, int64_t in, int64_t out, int experts, uint32_t box_y) {
  const cuuint64_t dims[3] = {(cuuint64_t)in, (cuuint64_t)out, (cuuint64_t)experts};
  const cuuint64_t strides[2] = {(cuuint64_t)in * 2, (cuuint64_t)in * 2 * (cuuint64_t)out};
  const cuuint32_t box[3] = {64, box_y, 1};
  return encode(m, base, 3, dims, strides, box);
}
// [expert][feature / 8][gate, up][feature % 8][in]: a box of 64 features
cudaError_t map_gated(CUtensorMap* m, const void* base, int64_t in, int64_t out, int experts) {
  const cuuint64_t row = (cuuint64_t)in * 2;
  const cuuint64_t dims[5] = {(cuuint64_t)in, 8, 2, (cuuint64_t)out / 16, (cuuint64_t)experts};
  const cuuint64_t strides[4] = {row, row * (cuuint64_t)(out / 2), row * 8, row * (cuuint64_t)out};
  const cuuint32_t box[5] = {64, 8, 2, 8, 1};
  return encode(m, base, 5, dims, strides, box);
}

template <typename T, int kMode, int kTok, bool kGated, bool kSplit = false>
cudaError_t allow_smem() {
  return cudaFuncSetAttribute(k_product<T, kMode, kTok, kGated, kSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Shape<kMode, kTok, kGated, kSplit>::kSmem);
}

template <typename T, int kMode, int kTok, bool kGated, bool kSplit = false>
cudaError_t launch(const char* name, const CUtensorMap& mf, const CUtensorMap& mt, const CUtensorMap& full, const Args& a,
                   int64_t grid, int cluster, int tiles_grad_w, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(Shape<kMode, kTok, kGated, kSplit>::kThreads);
  cfg.dynamicSmemBytes = Shape<kMode, kTok, kGated, kSplit>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  Launch guard(name, st);
  return cudaLaunchKernelEx(&cfg, k_product<T, kMode, kTok, kGated, kSplit>, mf, mt, full, a, tiles_grad_w);
}

// Forward and input gradient: the form by the mean number of rows of an expert
// that can have any, and by whether pairs would fill the GPU.  Measured (us,
// forward, 64 experts, 2048 -> 2048): 24 rows few 90, many 96; 48 rows few 104,
// many 98; 64 rows some 100, many 98; 128 rows some 102, many 108.  One matrix,
// few pairs: 40 rows 4096 -> 4096 many 31, few 23; 100 rows some 38, few 31; 512
// rows 2048 -> 2048 many 24, some 21.
template <typename T, int kMode, bool kGated>
cudaError_t launch_rows(const char* name, const CUtensorMap& mf, const void* x, int64_t x_stride, const Args& a, int sms,
                        cudaStream_t st) {
  const int64_t live = std::min<int64_t>(a.experts, a.rows);
  const int64_t mean = a.rows / std::max<int64_t>(1, live);
  // tiles: at most one ragged one per expert, and one behind the last
  auto bound = [&](int tok, int feat) {
    return (std::min<int64_t>(a.experts + 1, a.rows) + a.rows / tok) * ((a.feat + feat - 1) / feat);
  };
  constexpr int kWide = kGated ? 64 : 128;  // features of a block's tile
  const int64_t pairs = bound(256, 2 * kWide);
  CUtensorMap mt, full;
  cudaError_t e = map_rows(&mt, x, a.depth, a.rows, x_stride, kTokBox);
  if (e != cudaSuccess) return e;
  if (mean <= 32 || (mean <= 128 && 2 * pairs <= sms)) {
    const int64_t tiles = bound(32, kWide);
    const int chunks = (a.depth + kDepth - 1) / kDepth;
    int ranks = 1;
    while (ranks < 8 && tiles * ranks * 2 <= 2 * sms && chunks >= 8 * ranks) ranks *= 2;
    static_assert(kTokBox == 32, "a full tile is one small box");
    if (ranks == 1) return launch<T, kMode, 32, kGated>(name, mf, mt, mt, a, std::min<int64_t>(tiles, 2 * sms), 1, 0, st);
    return launch<T, kMode, 32, kGated, true>(name, mf, mt, mt, a, tiles * ranks, ranks, 0, st);
  }
  e = map_rows(&full, x, a.depth, a.rows, x_stride, 128);  // the tokens of a full tile, of one block
  if (e != cudaSuccess) return e;
  if (mean > 64 && (mean <= 128 || 4 * pairs <= sms))
    return launch<T, kMode, 128, kGated>(
        name, mf, mt, full, a, std::min<int64_t>(bound(128, kWide), sms), 1, 0, st);
  return launch<T, kMode, 256, kGated>(name, mf, mt, full, a, 2 * std::min<int64_t>(pairs, sms / 2), 2, 0, st);
}

Args base_args(const Product& p) {
  Args a{};
  a.rows = p.rows;
  a.experts = p.experts;
  a.activation = p.activation;
  a.offsets = p.offsets;
  a.y = p.y;
  a.y_stride = p.y_stride;
  a.status = p.status;
  a.polls = p.polls;
  a.starve = p.starve;
  return a;
}

template <typename T>
cudaError_t init_as() {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult got = cudaDriverEntryPointSymbolNotFound;
  cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &got);
  if (e != cudaSuccess) return e;
  if (!fn || got != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
  g_encode = reinterpret_cast<EncodeTiled>(fn);
  for (cudaError_t r : {allow_smem<T, kForward, 32, false>(), allow_smem<T, kForward, 32, true>(),
                        allow_smem<T, kForward, 32, false, true>(), allow_smem<T, kForward, 32, true, true>(),
                        allow_smem<T, kGradX, 32, false, true>(),
                        allow_smem<T, kForward, 128, false>(), allow_smem<T, kForward, 128, true>(),
                        allow_smem<T, kForward, 256, false>(), allow_smem<T, kForward, 256, true>(),
                        allow_smem<T, kGradX, 32, false>(), allow_smem<T, kGradX, 128, false>(),
                        allow_smem<T, kGradX, 256, false>(), allow_smem<T, kGradW, 256, false>()})
    if (r != cudaSuccess) return r;
  return cudaSuccess;
}

template <typename T>
cudaError_t fwd_as(const Product& p, int sms, cudaStream_t st) {
  const bool gated = p.activation == LAPSUM_ACT_SWIGLU;
  Args a = base_args(p);
  a.feat = (int)(gated ? p.out / 2 : p.out);
  a.depth = (int)p.in;
  a.bias = p.bias;
  a.residual = p.residual;
  a.residual_stride = p.residual_stride;
  a.preact = p.preact;
  a.preact_stride = p.preact_stride;
  CUtensorMap mf;
  const cudaError_t e = gated ? map_gated(&mf, p.weight, p.in, p.out, p.experts)
                        : map_weights(&mf, p.weight, p.in, p.out, p.experts, kLanes);
  if (e != cudaSuccess) return e;
  return gated ? launch_rows<T, kForward, true>("k_product_fwd", mf, p.x, p.x_stride, a, sms, st)
               : launch_rows<T, kForward, false>("k_product_fwd", mf, p.x, p.x_stride, a, sms, st);
}

template <typename T>
cudaError_t dx_as(const Product& p, int sms, cudaStream_t st) {
  Args a = base_args(p);
  a.feat = (int)p.in;
  a.depth = (int)p.out;
  CUtensorMap mf;
  const cudaError_t e = map_weights(&mf, p.weight, p.in, p.out, p.experts, kDepth);
  if (e != cudaSuccess) return e;
  return launch_rows<T, kGradX, false>("k_product_dx", mf, p.grad_h, p.grad_h_stride, a, sms, st);
}

template <typename T>
cudaError_t dweight_as(const Product& p, int sms, cudaStream_t st) {
  Args a = base_args(p);
  a.feat = (int)p.out;
  a.cols = (int)p.in;
  CUtensorMap mf, mt;
  cudaError_t e = map_rows(&mf, p.grad_h, p.out, p.rows, p.grad_h_stride, kDepth);
  if (e == cudaSuccess) e = map_rows(&mt, p.x, p.in, p.rows, p.x_stride, kDepth);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)p.experts * ((p.out + 255) / 256) * ((p.in + 255) / 256);
  return launch<T, kGradW, 256, false>("k_product_dw", mf, mt, mt, a, 2 * std::min<int64_t>(tiles, sms / 2), 2, (int)tiles, st);
}

}  // namespace
}  // namespace lapsum
