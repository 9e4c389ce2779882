// m2rnn_tc5.cuh -- 5th-generation tensor core (tcgen05), tensor memory and
// tensor-map copies, as inline PTX.
//
// Operand tiles lie in shared memory as the 128-byte-swizzled tensor-map copies
// leave them, in rows of 128 bytes, eight rows (1,024 bytes) to a swizzle atom:
//   * K-major: a row is one M/N index with 128 bytes of K.  SBO = 1,024 (eight
//     rows on); a step of 32 bytes along K moves the start address by 32.
//   * MN-major (bf16): a row is one K index with 64 M/N elements; a block of 64 K
//     rows is 8 KB and the next 64 M/N elements follow it.  LBO = 8,192 (64
//     elements on), SBO = 1,024 (eight K on); a step of 16 K moves the start by 2,048.
#pragma once
#include <cuda.h>

#include <cstdint>

#include "ptx.cuh"

namespace m2rnn {
namespace tc5 {

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Shared-memory descriptor with the 128-byte swizzle; lbo, sbo in bytes.
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}

// Instruction descriptor: fp32 accumulator; A, B both bf16 (kind::f16) or both e4m3
// (kind::f8f6f4, format 0).
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool e4m3, bool a_mn, bool b_mn) {
  return (1u << 4) | ((e4m3 ? 0u : 1u) << 7) | ((e4m3 ? 0u : 1u) << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// CG: 1, or 2 for a pair of CTAs (a cluster of two on neighbouring SMs) that work on one
// product: each holds half of A's rows, half of B's, and the accumulators of its rows.  The
// first CTA's thread issues for both; descriptors are offsets that hold in both.

// What becomes of an mma's A operand in the collector: read and forgotten, kept for the next mma, taken
// from there and kept, taken for the last time.
enum Keep { KEEP_NONE, KEEP_FILL, KEEP_USE, KEEP_LAST };

// D (+)= A B for one K step; one thread issues it.
template <bool E4M3, int CG, Keep K = KEEP_NONE>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool add) {
#define M2RNN_TC5_MMA(GROUP, KIND, COLLECT)                                                         \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                    \
               "tcgen05.mma.cta_group::" GROUP ".kind::" KIND COLLECT " [%0], %1, %2, %3, p;\n\t}" :: \
               "r"(d), "l"(a), "l"(b), "r"(id), "r"(static_cast<uint32_t>(add))                      \
               : "memory")
#define M2RNN_TC5_KEEP(GROUP, KIND)                              \
  if constexpr (K == KEEP_FILL)                                  \
    M2RNN_TC5_MMA(GROUP, KIND, ".collector::a::fill");           \
  else if constexpr (K == KEEP_USE)                              \
    M2RNN_TC5_MMA(GROUP, KIND, ".collector::a::use");            \
  else if constexpr (K == KEEP_LAST)                             \
    M2RNN_TC5_MMA(GROUP, KIND, ".collector::a::lastuse");        \
  else                                                           \
    M2RNN_TC5_MMA(GROUP, KIND, "")
  if constexpr (CG == 2) {
    if constexpr (E4M3) {
      M2RNN_TC5_KEEP("2", "f8f6f4");
    } else {
      M2RNN_TC5_KEEP("2", "f16");
    }
  } else {
    if constexpr (E4M3) {
      M2RNN_TC5_KEEP("1", "f8f6f4");
    } else {
      M2RNN_TC5_KEEP("1", "f16");
    }
  }
#undef M2RNN_TC5_KEEP
#undef M2RNN_TC5_MMA
}

// Arrives on `bar` (of both CTAs of a pair) when the thread's earlier mma have completed.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Tensor memory; one warp (of each CTA of a pair).
template <int CG>
__device__ __forceinline__ void alloc(uint32_t slot, uint32_t cols) {
  if constexpr (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void dealloc(uint32_t tm, uint32_t cols) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(cols) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(cols) : "memory");
}

// ---- pairs of CTAs -------------------------------------------------------------

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The address of a shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Hands over no memory (tensor memory whose loads have completed): a release would wait for
// the warp's global stores each time.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// ptx::mbar_wait on a barrier that the pair's other CTA arrives on too.
template <int CG>
__device__ __forceinline__ bool wait_released(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  if constexpr (CG == 1) return ptx::mbar_wait(bar, parity, limit_ns);
  const uint64_t t0 = ptx::globaltimer_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i) {
      uint32_t ok;
      asm volatile(
          "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(bar), "r"(parity)
          : "memory");
      if (ok) return true;
    }
    if (ptx::globaltimer_ns() - t0 > limit_ns) return false;
  }
}

// 32 columns of the warp's 32 lanes (one row per lane); wait_ld before they are used.
__device__ __forceinline__ void ld32(uint32_t ta, float (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
        "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
        "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
        "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(ta)
      : "memory");
}
// Completes the loads into r (named so that no use of r moves in front of it).
__device__ __forceinline__ void wait_ld(float (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                 "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]),
                 "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]),
                 "+f"(r[23]), "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]),
                 "+f"(r[30]), "+f"(r[31])::"memory");
}

// A box of a 3-dimensional tensor map into shared memory; its bytes are counted on `bar`
// (CG = 2: of either CTA of the pair).  x times the element's size is a multiple of 16.
template <int CG>
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Arrives on `bar` and announces `bytes`.
__device__ __forceinline__ void arrive_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

}  // namespace tc5
}  // namespace m2rnn
