// umma.cuh -- the tensor-core, tensor-memory and tiled-copy instructions of
// sm_100a that the experts' products use, one thin wrapper each.  Local
// copies only: no cluster multicast is ever issued.
#pragma once

#include <cuda.h>

#include "tma.cuh"

namespace lapsum {

// ---- tiled copies (one box of a tensor map into shared memory) --------------
// bar: shared-window address of the barrier that gets the bytes; kPair: the one
// of the pair's first block.
#define LAPSUM_TMA_LOAD(dims, coords, ...)                                                                          \
  do {                                                                                                              \
    if (kPair)                                                                                                      \
      asm volatile("cp.async.bulk.tensor." dims                                                                     \
                   ".shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, " coords      \
                   "], [%2];" ::"r"(smem_u32(dst)),                                                                 \
                   "l"(map), "r"(bar), __VA_ARGS__                                                                  \
                   : "memory");                                                                                     \
    else                                                                                                            \
      asm volatile("cp.async.bulk.tensor." dims                                                                     \
                   ".shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, " coords "], [%2];" ::"r"( \
                       smem_u32(dst)),                                                                              \
                   "l"(map), "r"(bar), __VA_ARGS__                                                                  \
                   : "memory");                                                                                     \
  } while (0)

template <bool kPair>
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  LAPSUM_TMA_LOAD("2d", "{%3, %4}", "r"(x), "r"(y));
}
template <bool kPair>
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  LAPSUM_TMA_LOAD("3d", "{%3, %4, %5}", "r"(x), "r"(y), "r"(z));
}
template <bool kPair>
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, int x, int y, int z, int u, int v,
                                            uint32_t bar) {
  LAPSUM_TMA_LOAD("5d", "{%3, %4, %5, %6, %7}", "r"(x), "r"(y), "r"(z), "r"(u), "r"(v));
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---- tensor memory ------------------------------------------------------------
// kPair: the two blocks of a cluster work as one on the products (all of these
// instructions of a kernel then take the pair form).  One whole warp each; cols
// a power of two, 32..512.
template <bool kPair>
__device__ __forceinline__ void tmem_alloc(uint32_t* where, uint32_t cols) {
  if (kPair) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(where)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(where)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}
template <bool kPair>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  if (kPair)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
// 16 lanes x 32 columns as four 16 x 8 fragments: with r = lane / 4 and
// c = 2 (lane % 4), v[4 j + 0 / 1] is row r, columns 8 j + c / + 1 and
// v[4 j + 2 / 3] the same of row r + 8
__device__ __forceinline__ void tmem_load_16x32(uint32_t addr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// ---- 8 x 8 fragments of 16-bit values between registers and shared memory ---------
// Lane l gives the address of row l % 8 of matrix l / 8 (16 bytes); register m of
// lane l holds row l / 4, columns 2 (l % 4) and + 1 of matrix m (rows and columns
// change places in the transposing forms).
template <bool kTrans>
__device__ __forceinline__ void stage_4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  if (kTrans)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
  else
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ void fetch_4_trans(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float lds4(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// ---- matrix products --------------------------------------------------------------
// Shared-memory operand in the 128-byte swizzle that a tiled copy writes.
// Along the contraction contiguous ("K major"): rows of 64 values (128 bytes),
// 8 rows make a swizzle atom of 1024 bytes; a step of 16 along the contraction
// moves the address by 32 bytes.  Along the other axis contiguous ("MN major"):
// blocks of 64 values x depth, one 128-byte line per index of the contraction;
// lead is the distance between such blocks, a step of 16 moves by 2048 bytes.
__device__ __forceinline__ uint64_t operand_desc(uint32_t smem_addr, uint32_t lead_bytes) {
  return (uint64_t)((smem_addr >> 4) & 0x3FFFu) | ((uint64_t)(lead_bytes >> 4) << 16) |
         ((uint64_t)(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// kind::f16 with fp32 accumulators: both operands bf16 (or both fp16)
__host__ __device__ constexpr uint32_t instr_desc(bool bf16, bool a_mn_major, bool b_mn_major, uint32_t m,
                                                  uint32_t n) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn_major ? 1u : 0u) << 15) |
         ((b_mn_major ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
// D[tmem] (+)= A B for one step of 16 along the contraction; one thread issues.
// kPair: the first block of the pair issues for both; each holds its own half
// of A's rows and of the accumulator's, and half of B's
template <bool kPair>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  if (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}
// The barrier gets one arrival when all products issued so far are done; kPair:
// the barrier of that place in both blocks does.
template <bool kPair>
__device__ __forceinline__ void mma_commit(uint64_t* mbar) {
  if (kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(mbar)),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(mbar))
                 : "memory");
}

// ---- clusters ------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// v to this block's shared address `addr`, in block `rank`
__device__ __forceinline__ void cluster_store(uint32_t addr, uint32_t rank, float v) {
  uint32_t there;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(addr), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there), "f"(v) : "memory");
}

// the shared-window address of this block's `p` in block `rank`
__device__ __forceinline__ uint32_t in_block(const void* p, uint32_t rank) {
  uint32_t there;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(smem_u32(p)), "r"(rank));
  return there;
}
// One arrival at a barrier of the cluster.  kRelease orders this thread's
// ordinary writes before it; copies and reads of tensor memory need no such
// order, and it is far from free.
template <bool kRelease>
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  if (kRelease)
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
  else
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void arrive_expect_at(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
// its counterpart, a poll after which what the other block's releasing arrival
// ordered is visible
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* mbar, uint32_t phase) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(mbar)), "r"(phase)
      : "memory");
  return ok != 0u;
}

}  // namespace lapsum
