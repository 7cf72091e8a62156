// Inline-PTX building blocks of the training-block kernels beyond those of
// sm103_ptx.cuh: waits that suspend, pairs of blocks on one product
// (cta_group::2), TMEM loads in the fragment layout.  Each is written from the
// public PTX ISA description of its instruction.  (A file of its own: the
// attention kernels' committed counters hold for sm103_ptx.cuh as it is.)
#pragma once
#include "sm103_ptx.cuh"

namespace detattn {

// ---------------------------------------------------------------- waits
// Whether the phase with the given parity has completed; never suspends.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// mbar_wait with a hint that lets the hardware suspend the thread for up to 20
// us at a time (it wakes when the phase completes), so that warps that wait
// long take no issue slots from those at work; and for a barrier that threads
// of another block of the cluster arrive on, whose earlier writes are visible
// after the wait.
template <bool CLUSTER>
__device__ __forceinline__ bool mbar_try_wait_hint(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (CLUSTER)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, 20000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  return ok != 0;
}
template <bool CLUSTER = false>
__device__ __forceinline__ bool mbar_wait_hint(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  if (mbar_try_wait_hint<CLUSTER>(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  for (uint32_t it = 0; it < (1u << 26); ++it) {
    if (mbar_try_wait_hint<CLUSTER>(bar, parity)) return true;
    if (globaltimer_ns() - t0 > limit_ns) return false;
  }
  return false;
}

// ---- CTA pairs (cta_group::2): two blocks of a cluster whose ranks differ in
// the last bit work on one product of up to 256 rows.  Both allocate (and
// free) their TMEM together, the even block issues, each block's shared memory
// holds its half of the rows of A and of the columns of B at the same offsets,
// and each block's TMEM receives its half of the rows.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void mma_ss_x4_pair(uint32_t d_tmem, uint64_t a0, uint64_t a1, uint64_t a2,
                                               uint64_t a3, uint64_t b0, uint64_t b1, uint64_t b2,
                                               uint64_t b3, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %10, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %5, %9, p;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %2, %6, %9, 1;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %3, %7, %9, 1;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %4, %8, %9, 1;\n\t}" ::"r"(d_tmem),
      "l"(a0), "l"(a1), "l"(a2), "l"(a3), "l"(b0), "l"(b1), "l"(b2), "l"(b3), "r"(idesc),
      "r"(accumulate)
      : "memory");
}
// One arrival on the barrier at this offset in both blocks of the pair.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;\n\t}" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// A load into this block's shared memory that completes on a barrier of either
// block of the pair (`bar`: a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                                 int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
// Arrival on an mbarrier of a block of the pair (`bar` from map_shared_rank) by
// a thread whose writes are to its own block's shared memory and already
// behind a fence.proxy.async: the other block only learns that its products
// may start, and each tensor core reads its own block's memory.  Releasing to
// the cluster instead (mbar_arrive_remote) waits for everything the thread's
// SM has under way; at one arrival a step that took the weight gradient of
// 8192 x 4096 x 6144 from 296 to 655 us.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// ---------------------------------------------------------------- TMEM
// 16 lanes x 256 bits, twice (sixteen columns): thread i gets columns
// 2 (i % 4), + 1 of lane i / 4 in r[0], r[1], of lane i / 4 + 8 in r[2], r[3],
// and the same of the next eight columns in r[4] .. r[7].
__device__ __forceinline__ void tmem_ld_16x256b_x2_nowait(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : DETATTN_R8(r, 0)
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void reg_fence8(uint32_t (&r)[8]) {
  asm volatile("" : DETATTN_RW8(r, 0) : : "memory");
}

// ---------------------------------------------------------------- misc
// 1 / x within 2^-23; beyond 2^126 zero.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace detattn
