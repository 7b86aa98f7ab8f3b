// Pairs of CTAs that issue tcgen05 work together (cta_group::2): the first CTA
// of a cluster of two, the leader, issues the MMAs for both, each CTA holding
// half of A's rows, half of B and half of D.  M = 128 puts rows 0..63 of D in
// the leader and 64..127 in the other: in each, lane l < 64 holds row l's first
// N / 2 columns and lane l + 64 its others.
#pragma once

#include "sm103_ptx.cuh"

namespace mla {

// Warp-wide, in both CTAs.
__device__ __forceinline__ void pair_tmem_alloc(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// The words of a shared-memory matrix descriptor: the low one moves with the address
// (in units of 16 bytes), the high one does not.
struct MatrixWords {
  uint32_t lo, hi;
  __device__ __forceinline__ MatrixWords(const void* smem, uint32_t lbo_bytes, uint32_t sbo_bytes) {
    const uint64_t d = make_smem_desc(smem_u32(smem), lbo_bytes, sbo_bytes, kSmemLayoutSW128);
    lo = static_cast<uint32_t>(d);
    hi = static_cast<uint32_t>(d >> 32);
  }
};

// D (+)= A B over both CTAs' halves.  Called by a whole warp of the leader, converged,
// of which one thread issues: with every operand the same across the warp the
// addresses stay in uniform registers (from inside a branch that one thread takes,
// an MMA took 80-90 cycles to issue, two and a half times what it runs).
__device__ __forceinline__ void pair_mma_bf16(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                              uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 a, b;\n setp.ne.b32 p, %6, 0;\n"
      " mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n}" ::"r"(d_tmem),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on `bar` of both CTAs once the warp's MMAs so far have completed.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Arrive on the barrier at `addr` (mapa_shared) of a CTA of the cluster.  What the
// arrival announces is in this CTA's shared or tensor memory, where the pair's MMAs
// read it: it is ordered before by fence.proxy.async or tcgen05.fence, and a
// release to the whole cluster, which waits for every access of the thread, costs
// 1,200 cycles here.
__device__ __forceinline__ void cluster_mbar_arrive(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// As mbar_wait for roles on the path of every tile: no sleep between looks, and the
// clock, whose reading takes longer than most of these waits, is looked at only
// after some hundred of them.
__device__ __forceinline__ bool pair_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  uint64_t t0 = 0;
  for (uint32_t n = 1;; ++n) {
    if (mbar_test(bar, parity)) return true;
    if ((n & 255u) == 0) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (*abort || now - t0 > limit_ns) return false;
    }
  }
}

// Tile loads of one CTA whose bytes count on the barrier at bar_addr (mapa_shared)
// of either CTA of the pair.
__device__ __forceinline__ void pair_tma_load_3d(void* dst, const CUtensorMap* map, uint32_t bar_addr, int32_t x,
                                                 int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_addr), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void pair_tma_gather4(void* dst, const CUtensorMap* map, uint32_t bar_addr, int32_t x,
                                                 const int32_t (&row)[4]) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_addr), "r"(x), "r"(row[0]), "r"(row[1]), "r"(row[2]), "r"(row[3])
      : "memory");
}

}  // namespace mla
