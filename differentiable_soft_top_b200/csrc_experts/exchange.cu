// exchange.cu -- between token order and expert order: the plan (a stable
// counting sort of the slots by expert), the gather of token rows and the
// weighted sum back, each with its gradient.
//
// All but the plan are bound by memory: 16 bytes per lane and access where the
// addresses allow it, 8 accesses of a lane in flight.  Measured at 4096 tokens x
// 8 x 2048, bf16, in a graph, inputs larger than L2: dispatch 29 us (5.3 TB/s),
// weighted sum 31 (4.9), with a residual 37 (4.6), its gradient 47 (6.1); plan of
// those 32768 slots 8.  For short batches dispatch splits a row over several warps
// so that the GPU is full; the weighted sum has at most a block per token, its
// gradient a warp per slot.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "chain.cuh"
#include "experts.h"

namespace lapsum {
namespace {

// ---- the plan ---------------------------------------------------------------------
// A block sorts a range of `per` slots.  First kernel: a histogram per block.
// Second: every block adds the histograms before its own and in all (at most
// kMaxBlocks of them, one thread per expert), scans the experts, and places
// its slots: each warp a contiguous part, 32 slots at a time in ascending
// order, equal experts ranked by match_any.  Integer counts only.
constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kMaxBlocks = 256;

struct PlanShape {
  int per, blocks;
};
PlanShape plan_shape(int64_t slots) {
  // one block up to 4096 slots (one launch), then 2048 per block until there
  // are kMaxBlocks
  PlanShape p;
  int64_t per = slots <= 4096 ? 4096 : std::max<int64_t>(2048, (slots + kMaxBlocks - 1) / kMaxBlocks);
  per = (per + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
  p.per = (int)per;
  p.blocks = (int)((slots + per - 1) / per);
  return p;
}

__global__ void __launch_bounds__(kPlanThreads) k_plan_count(const int32_t* chosen, int64_t slots, int experts, int per,
                                                             int32_t* hist) {
  grid_launch_next();
  __shared__ int cnt[LAPSUM_EXPERTS_MAX];
  for (int e = threadIdx.x; e < experts; e += kPlanThreads) cnt[e] = 0;
  grid_wait_previous();
  __syncthreads();
  const int64_t s0 = (int64_t)blockIdx.x * per, s1 = min(slots, s0 + per);
  for (int64_t s = s0 + threadIdx.x; s < s1; s += kPlanThreads) {
    const int e = __ldg(chosen + s);
    if ((unsigned)e < (unsigned)experts) atomicAdd(cnt + e, 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < experts; e += kPlanThreads) hist[(int64_t)blockIdx.x * experts + e] = cnt[e];
}

// hist == null: one block holds all slots
__global__ void __launch_bounds__(kPlanThreads) k_plan_place(const int32_t* chosen, int64_t slots, int experts, int per,
                                                             const int32_t* hist, int32_t* offsets, int32_t* rows,
                                                             int32_t* slot_of) {
  grid_launch_next();
  extern __shared__ int sh[];
  int* total = sh;                       // [experts]
  int* start = sh + experts;             // [experts] first row of this block's slots of an expert
  int* mine = sh + 2 * experts;          // [warps][experts]
  __shared__ int chunk[kPlanWarps + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t s0 = (int64_t)blockIdx.x * per, s1 = min(slots, s0 + per);
  for (int i = threadIdx.x; i < kPlanWarps * experts; i += kPlanThreads) mine[i] = 0;
  grid_wait_previous();
  __syncthreads();
  const int64_t part = per / kPlanWarps;  // a multiple of 32
  const int64_t w0 = s0 + warp * part, w1 = min(s1, w0 + part);
  int* cnt = mine + warp * experts;
  for (int64_t s = w0 + lane; s < w1; s += 32) {
    const int e = __ldg(chosen + s);
    if ((unsigned)e < (unsigned)experts) atomicAdd(cnt + e, 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < experts; e += kPlanThreads) {
    int run = 0;
    for (int w = 0; w < kPlanWarps; ++w) {  // counts to starts within the block
      const int c = mine[w * experts + e];
      mine[w * experts + e] = run;
      run += c;
    }
    int before = 0, all = run;
    if (hist) {
      all = 0;
#pragma unroll 8
      for (int b = 0; b < (int)gridDim.x; ++b) {
        const int c = __ldg(hist + (int64_t)b * experts + e);
        before += b < (int)blockIdx.x ? c : 0;
        all += c;
      }
    }
    total[e] = all;
    start[e] = before;
  }
  __syncthreads();
  // exclusive scan over the experts: kPlanThreads at a time
  int base = 0;
  for (int e0 = 0; e0 < experts; e0 += kPlanThreads) {
    const int e = e0 + threadIdx.x;
    const int own = e < experts ? total[e] : 0;
    int v = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += u;
    }
    if (lane == 31) chunk[warp] = v;
    __syncthreads();
    int add = base;
    for (int w = 0; w < warp; ++w) add += chunk[w];
    int sum = 0;
    for (int w = 0; w < kPlanWarps; ++w) sum += chunk[w];
    if (e < experts) {
      const int first = add + v - own;
      start[e] += first;
      if (blockIdx.x == 0) offsets[e] = first;
    }
    base += sum;
    __syncthreads();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) offsets[experts] = base;
  // rows nobody owns
  for (int64_t r = max(s0, (int64_t)base) + threadIdx.x; r < s1; r += kPlanThreads) slot_of[r] = -1;
  for (int64_t g = w0; g < w1; g += 32) {
    const int64_t s = g + lane;
    int e = s < w1 ? __ldg(chosen + s) : -1;
    if ((unsigned)e >= (unsigned)experts) e = -1;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    int row = -1;
    if (e >= 0) row = start[e] + cnt[e] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (e >= 0 && (same >> lane) == 1u) cnt[e] += __popc(same);  // the highest lane of its expert
    __syncwarp();
    if (s < w1) {
      rows[s] = row;
      if (row >= 0) slot_of[row] = (int)s;
    }
  }
}

// ---- rows ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;

template <int kDtype>
struct Elem;
template <>
struct Elem<LAPSUM_F32> {
  using T = float;
  static __device__ __forceinline__ float get(T v) { return v; }
  static __device__ __forceinline__ T put(float v) { return v; }
};
template <>
struct Elem<LAPSUM_BF16> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float get(T v) { return __bfloat162float(v); }
  static __device__ __forceinline__ T put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<LAPSUM_F16> {
  using T = __half;
  static __device__ __forceinline__ float get(T v) { return __half2float(v); }
  static __device__ __forceinline__ T put(float v) { return __float2half_rn(v); }
};

// kVec values moved together: 16 bytes, or one value where some address does
// not lie on a 16-byte boundary
template <int kDtype, int kVec>
struct alignas(kVec * sizeof(typename Elem<kDtype>::T)) Pack {
  typename Elem<kDtype>::T v[kVec];
};
template <int kDtype>
constexpr int full_vec() {
  return 16 / (int)sizeof(typename Elem<kDtype>::T);
}

// the pack's values in fp32; 16-bit pairs are taken apart as words
template <int kDtype, int kVec>
__device__ __forceinline__ void unpack(const Pack<kDtype, kVec>& p, float (&f)[kVec]) {
  if constexpr (kVec == 1 || kDtype == LAPSUM_F32) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) f[i] = Elem<kDtype>::get(p.v[i]);
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(p.v);
#pragma unroll
    for (int i = 0; i < kVec / 2; ++i) {
      if constexpr (kDtype == LAPSUM_BF16) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(w + i));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
      }
    }
  }
}
template <int kDtype, int kVec>
__device__ __forceinline__ Pack<kDtype, kVec> pack(const float (&f)[kVec]) {
  Pack<kDtype, kVec> p;
  if constexpr (kVec == 1 || kDtype == LAPSUM_F32) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) p.v[i] = Elem<kDtype>::put(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kVec / 2; ++i) {
      if constexpr (kDtype == LAPSUM_BF16)
        reinterpret_cast<__nv_bfloat162*>(p.v)[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      else
        reinterpret_cast<__half2*>(p.v)[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    }
  }
  return p;
}

template <int kDtype, int kVec>
__device__ __forceinline__ Pack<kDtype, kVec> zero_pack() {
  Pack<kDtype, kVec> p;
#pragma unroll
  for (int i = 0; i < kVec; ++i) p.v[i] = Elem<kDtype>::put(0.0f);
  return p;
}

// The unit of work: warp `unit` takes part `unit % parts` of row `unit / parts`.
struct Units {
  int64_t rows;
  int parts;
  int per;  // packs per part
  int packs;
};

template <int kDtype, int kVec>
__global__ void __launch_bounds__(kRowThreads) k_dispatch(const typename Elem<kDtype>::T* __restrict__ x,
                                                          int64_t x_stride, const int32_t* __restrict__ slot_of, int k,
                                                          typename Elem<kDtype>::T* __restrict__ out, int64_t out_stride,
                                                          int64_t slots, Units u) {
  using P = Pack<kDtype, kVec>;
  grid_launch_next();
  grid_wait_previous();
  const int lane = threadIdx.x & 31;
  const int64_t nwarp = (int64_t)gridDim.x * (kRowThreads / 32);
  for (int64_t w = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); w < u.rows * u.parts; w += nwarp) {
    const int64_t r = w / u.parts;
    const int p0 = (int)(w - r * u.parts) * u.per, p1 = min(u.packs, p0 + u.per);
    const int s = __ldg(slot_of + r);
    const bool some = (uint64_t)(int64_t)s < (uint64_t)slots;
    const P* src = reinterpret_cast<const P*>(x + (some ? s / k : 0) * x_stride);
    P* dst = reinterpret_cast<P*>(out + r * out_stride);
    for (int p = p0 + lane; p < p1; p += 256) {
      P v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = src[min(p + 32 * i, p1 - 1)];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (p + 32 * i < p1) dst[p + 32 * i] = some ? v[i] : zero_pack<kDtype, kVec>();
    }
  }
}

// `per_row` threads (32 .. 256, a power of two) take a token; each keeps kPacks
// accesses of kRows rows in flight, 8 in all whatever k.  A row is read in pieces
// as long as the block allows: DRAM likes 4 KB of a row at once (a warp per
// token, which came back for 512 bytes of each row at a time, took 1.3 to 2
// times as long).  The next token's row numbers are read ahead; the grid is what
// is resident (8 blocks per SM of work in turn: 43 us, 2: 41, 4096 x 8 x 2048 with
// a residual, between events).
template <int kDtype, int kVec, int kRows, int kPacks>
__global__ void __launch_bounds__(kRowThreads, 2)
    k_combine(const typename Elem<kDtype>::T* __restrict__ y, int64_t y_stride, const float* __restrict__ weights,
              const int32_t* __restrict__ rows, int64_t tokens, int k, int64_t all_rows,
              const typename Elem<kDtype>::T* __restrict__ residual, int64_t res_stride,
              typename Elem<kDtype>::T* __restrict__ out, int64_t out_stride, int packs, int per_row) {
  using P = Pack<kDtype, kVec>;
  grid_launch_next();
  grid_wait_previous();
  const int in_block = kRowThreads / per_row;
  const int64_t step = (int64_t)gridDim.x * in_block;
  int64_t t = (int64_t)blockIdx.x * in_block + threadIdx.x / per_row;
  auto look = [&](int64_t tok, int j0, int (&r)[kRows]) {
#pragma unroll
    for (int j = 0; j < kRows; ++j) r[j] = __ldg(rows + tok * k + min(j0 + j, k - 1));
  };
  int r[kRows], r1[kRows];
  if (t < tokens) look(t, 0, r1);
  for (; t < tokens; t += step) {
#pragma unroll
    for (int j = 0; j < kRows; ++j) r[j] = r1[j];
    if (t + step < tokens) look(t + step, 0, r1);
    for (int p = threadIdx.x % per_row; p < packs; p += per_row * kPacks) {
      float acc[kPacks][kVec];
#pragma unroll
      for (int q = 0; q < kPacks; ++q) {
        P v = zero_pack<kDtype, kVec>();
        if (residual) v = reinterpret_cast<const P*>(residual + t * res_stride)[min(p + q * per_row, packs - 1)];
        unpack<kDtype, kVec>(v, acc[q]);
      }
      for (int j0 = 0; j0 < k; j0 += kRows) {
        if (k > kRows) look(t, j0, r);
        // all loads first, without a branch between them (places behind the last
        // repeat it and are not added)
        P v[kRows][kPacks];
        float c[kRows];
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          const P* src = reinterpret_cast<const P*>(y + ((uint64_t)(int64_t)r[j] < (uint64_t)all_rows ? (int64_t)r[j] : 0) * y_stride);
#pragma unroll
          for (int q = 0; q < kPacks; ++q) v[j][q] = src[min(p + q * per_row, packs - 1)];
        }
#pragma unroll
        for (int j = 0; j < kRows; ++j) c[j] = weights ? __ldg(weights + t * k + min(j0 + j, k - 1)) : 1.0f;
#pragma unroll
        for (int j = 0; j < kRows; ++j)
          if (j0 + j < k) {
            const bool some = (uint64_t)(int64_t)r[j] < (uint64_t)all_rows;
#pragma unroll
            for (int q = 0; q < kPacks; ++q) {
              if (!some) v[j][q] = zero_pack<kDtype, kVec>();  // a row that is not there adds w * 0
              float f[kVec];
              unpack<kDtype, kVec>(v[j][q], f);
#pragma unroll
              for (int i = 0; i < kVec; ++i) acc[q][i] = fmaf(c[j], f[i], acc[q][i]);
            }
          }
      }
#pragma unroll
      for (int q = 0; q < kPacks; ++q)
        if (p + q * per_row < packs) {
          reinterpret_cast<P*>(out + t * out_stride)[p + q * per_row] = pack<kDtype, kVec>(acc[q]);
        }
    }
  }
}

// One warp per slot: dY of its row and <g, y>.  Row numbers without a slot are
// those a warp of the same number clears.
template <int kDtype, int kVec>
__global__ void __launch_bounds__(kRowThreads)
    k_combine_bwd(const typename Elem<kDtype>::T* __restrict__ g, int64_t g_stride,
                  const typename Elem<kDtype>::T* __restrict__ y, int64_t y_stride, const float* __restrict__ weights,
                  const int32_t* __restrict__ rows, const int32_t* __restrict__ slot_of, int k, int64_t slots,
                  typename Elem<kDtype>::T* __restrict__ gy, int64_t gy_stride, float* __restrict__ gw, int packs) {
  using P = Pack<kDtype, kVec>;
  grid_launch_next();
  grid_wait_previous();
  const int lane = threadIdx.x & 31;
  const int64_t nwarp = (int64_t)gridDim.x * (kRowThreads / 32);
  for (int64_t s = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); s < slots; s += nwarp) {
    int row = __ldg(rows + s);
    if ((uint64_t)(int64_t)row >= (uint64_t)slots) row = -1;
    const float wt = weights ? __ldg(weights + s) : 1.0f;
    // row number s has no slot: none in range, or one whose place was taken away
    const int from = gy ? __ldg(slot_of + s) : 0;
    const bool some = (uint64_t)(int64_t)from < (uint64_t)slots;
    const int back = __ldg(rows + (some ? from : 0));
    float dot = 0.0f;
    if (row >= 0) {
      const P* gp = reinterpret_cast<const P*>(g + s / k * g_stride);
      const P* yp = reinterpret_cast<const P*>(y + (int64_t)row * y_stride);
      P* op = reinterpret_cast<P*>(gy + (int64_t)row * gy_stride);
      for (int p = lane; p < packs; p += 128) {
        P a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          a[i] = gp[min(p + 32 * i, packs - 1)];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (gw) b[i] = yp[min(p + 32 * i, packs - 1)];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (p + 32 * i < packs) {
            float f[kVec];
            unpack<kDtype, kVec>(a[i], f);
            if (gw) {
              float h[kVec];
              unpack<kDtype, kVec>(b[i], h);
#pragma unroll
              for (int q = 0; q < kVec; ++q) dot = fmaf(f[q], h[q], dot);
            }
#pragma unroll
            for (int q = 0; q < kVec; ++q) f[q] *= wt;
            if (gy) op[p + 32 * i] = pack<kDtype, kVec>(f);
          }
      }
    }
    if (gw) {
#pragma unroll
      for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
      if (lane == 0) gw[s] = dot;
    }
    if (gy && (!some || back != (int)s)) {
      P* op = reinterpret_cast<P*>(gy + s * gy_stride);
      for (int p = lane; p < packs; p += 32) op[p] = zero_pack<kDtype, kVec>();
    }
  }
}

bool on16(const void* p, int64_t stride, int size) {
  return !p || (!((uintptr_t)p & 15u) && !((stride * size) & 15));
}

Units make_units(int64_t rows, int64_t packs, int sms) {
  Units u;
  u.rows = rows;
  u.packs = (int)packs;
  // about 32 warps per SM, each with at least one access of all its lanes
  const int64_t want = std::max<int64_t>(1, (int64_t)sms * 32 / std::max<int64_t>(1, rows));
  const int64_t most = std::max<int64_t>(1, (packs + 31) / 32);
  u.per = (int)((((packs + std::min(want, most) - 1) / std::min(want, most)) + 31) / 32 * 32);
  u.parts = (int)((packs + u.per - 1) / u.per);
  return u;
}
unsigned grid_of(int64_t warps, int sms) {
  const int64_t blocks = (warps + kRowThreads / 32 - 1) / (kRowThreads / 32);
  return (unsigned)std::max<int64_t>(1, std::min<int64_t>(blocks, (int64_t)sms * 64));
}

template <int kDtype, int kVec>
void dispatch_as(const void* x, int64_t tokens, int k, int64_t dim, int64_t x_stride, const int32_t* slot_of, void* out,
                 int64_t out_stride, int sms, cudaStream_t st) {
  using T = typename Elem<kDtype>::T;
  const Units u = make_units(tokens * k, dim / kVec, sms);
  launch_ex(true, k_dispatch<kDtype, kVec>, dim3(grid_of(u.rows * u.parts, sms)), dim3(kRowThreads), 0, st,
      static_cast<const T*>(x), x_stride, slot_of, k, static_cast<T*>(out), out_stride, tokens * k, u);
}
template <int kDtype, int kVec>
void combine_as(const void* y, int64_t tokens, int k, int64_t dim, int64_t y_stride, const float* weights,
                const int32_t* rows, const void* residual, int64_t res_stride, void* out, int64_t out_stride, int sms,
                cudaStream_t st) {
  using T = typename Elem<kDtype>::T;
  const int packs = (int)(dim / kVec), each = k <= 2 ? 4 : k <= 4 ? 2 : 1;
  int per_row = 32;
  while (per_row < kRowThreads && per_row * each < packs) per_row *= 2;
  const int64_t blocks = (tokens + kRowThreads / per_row - 1) / (kRowThreads / per_row);
  auto* kernel = k <= 2 ? k_combine<kDtype, kVec, 2, 4> : k <= 4 ? k_combine<kDtype, kVec, 4, 2> : k_combine<kDtype, kVec, 8, 1>;
  launch_ex(true, kernel, dim3((unsigned)std::min<int64_t>(blocks, (int64_t)sms * 2)), dim3(kRowThreads), 0, st,
      static_cast<const T*>(y), y_stride, weights, rows, tokens, k, tokens * k, static_cast<const T*>(residual), res_stride,
      static_cast<T*>(out), out_stride, packs, per_row);
}
template <int kDtype, int kVec>
void combine_bwd_as(const void* grad, int64_t tokens, int k, int64_t dim, int64_t grad_stride, const void* y,
                    int64_t y_stride, const float* weights, const int32_t* rows, const int32_t* slot_of, void* grad_y,
                    int64_t grad_y_stride, float* grad_weights, int sms, cudaStream_t st) {
  using T = typename Elem<kDtype>::T;
  launch_ex(true, k_combine_bwd<kDtype, kVec>, dim3(grid_of(tokens * k, sms)), dim3(kRowThreads), 0, st,
      static_cast<const T*>(grad), grad_stride, static_cast<const T*>(y), y_stride, weights, rows, slot_of, k,
      tokens * k, static_cast<T*>(grad_y), grad_y_stride, grad_weights, (int)(dim / kVec));
}

}  // namespace

size_t plan_workspace(int64_t slots, int experts) {
  const PlanShape p = plan_shape(slots);
  return p.blocks > 1 ? (((size_t)p.blocks * experts * 4 + 255) & ~size_t(255)) : 0;
}

cudaError_t launch_plan(const int32_t* chosen, int64_t slots, int experts, int32_t* offsets, int32_t* rows,
                        int32_t* slot_of, void* ws, cudaStream_t st) {
  const PlanShape p = plan_shape(slots);
  int32_t* hist = p.blocks > 1 ? static_cast<int32_t*>(ws) : nullptr;
  if (hist) {
    Launch guard("k_plan_count", st);
    launch_ex(true, k_plan_count, dim3(p.blocks), dim3(kPlanThreads), 0, st, chosen, slots, experts, p.per, hist);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  Launch guard("k_plan_place", st);
  launch_ex(true, k_plan_place, dim3(p.blocks), dim3(kPlanThreads), (size_t)(2 + kPlanWarps) * experts * 4, st, chosen, slots,
            experts, p.per, (const int32_t*)hist, offsets, rows, slot_of);
  return cudaGetLastError();
}

cudaError_t exchange_init() {
  return cudaFuncSetAttribute(k_plan_place, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (2 + kPlanWarps) * LAPSUM_EXPERTS_MAX * 4);
}

#define LAPSUM_BY_DTYPE(fn, vec, ...)                                             \
  do {                                                                            \
    if (dtype == LAPSUM_F32) {                                                    \
      vec ? fn<LAPSUM_F32, full_vec<LAPSUM_F32>()>(__VA_ARGS__) : fn<LAPSUM_F32, 1>(__VA_ARGS__);    \
    } else if (dtype == LAPSUM_BF16) {                                            \
      vec ? fn<LAPSUM_BF16, full_vec<LAPSUM_BF16>()>(__VA_ARGS__) : fn<LAPSUM_BF16, 1>(__VA_ARGS__); \
    } else {                                                                      \
      vec ? fn<LAPSUM_F16, full_vec<LAPSUM_F16>()>(__VA_ARGS__) : fn<LAPSUM_F16, 1>(__VA_ARGS__);    \
    }                                                                             \
  } while (0)

cudaError_t launch_dispatch(const void* x, int dtype, int64_t tokens, int k, int64_t dim, int64_t x_stride,
                            const int32_t* slot_of, void* out, int64_t out_stride, int sms, cudaStream_t st) {
  const int z = dtype == LAPSUM_F32 ? 4 : 2;
  const bool vec = on16(x, x_stride, z) && on16(out, out_stride, z) && dim * z % 16 == 0;
  Launch guard("k_dispatch", st);
  LAPSUM_BY_DTYPE(dispatch_as, vec, x, tokens, k, dim, x_stride, slot_of, out, out_stride, sms, st);
  return cudaGetLastError();
}

cudaError_t launch_combine(const void* y, int dtype, int64_t tokens, int k, int64_t dim, int64_t y_stride,
                           const float* weights, const int32_t* rows, const void* residual, int64_t res_stride,
                           void* out, int64_t out_stride, int sms, cudaStream_t st) {
  const int z = dtype == LAPSUM_F32 ? 4 : 2;
  const bool vec = on16(y, y_stride, z) && on16(out, out_stride, z) && on16(residual, res_stride, z) && dim * z % 16 == 0;
  Launch guard("k_combine", st);
  LAPSUM_BY_DTYPE(combine_as, vec, y, tokens, k, dim, y_stride, weights, rows, residual, res_stride, out, out_stride,
                  sms, st);
  return cudaGetLastError();
}

cudaError_t launch_combine_bwd(const void* grad, int dtype, int64_t tokens, int k, int64_t dim, int64_t grad_stride,
                               const void* y, int64_t y_stride, const float* weights, const int32_t* rows,
                               const int32_t* slot_of, void* grad_y, int64_t grad_y_stride, float* grad_weights,
                               int sms, cudaStream_t st) {
  const int z = dtype == LAPSUM_F32 ? 4 : 2;
  const bool vec = on16(grad, grad_stride, z) && on16(y, y_stride, z) && on16(grad_y, grad_y_stride, z) && dim * z % 16 == 0;
  Launch guard("k_combine_bwd", st);
  LAPSUM_BY_DTYPE(combine_bwd_as, vec, grad, tokens, k, dim, grad_stride, y, y_stride, weights, rows, slot_of, grad_y,
                  grad_y_stride, grad_weights, sms, st);
  return cudaGetLastError();
}

}  // namespace lapsum
