// Inline-PTX wrappers for a CTA pair (cta_group::2): one tcgen05.mma over two SMs' shared memory
// and TMEM, TMA loads that count on the leader's barrier (never multicast), and the cluster's
// barrier.  Written from the PTX ISA (tcgen05, cp.async.bulk.tensor, mbarrier, mapa sections).
#pragma once

#include "tc_ptx.cuh"

namespace dsv4 {
namespace tc {

__device__ __forceinline__ uint32_t cluster_cta_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The address, in the cluster's shared window, of the same variable in CTA `rank`.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// One box of a tensor into this CTA's shared memory; the bytes count on the barrier at `bar`
// (an address in the cluster's window, in either CTA of the pair).  Returns whether the phase of `next`
// is complete: asked for ahead of the load and looked at behind it.
__device__ __forceinline__ bool tma2_load_2d_test(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar,
                                                  uint64_t* next, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred r;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 r, [%6], %7;\n\t"
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%1], [%2, {%3, %4}], [%5];\n\t"
      "selp.u32 %0, 1, 0, r;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(smem_u32(next)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool tma2_load_3d_test(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar,
                                                  uint64_t* next, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred r;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 r, [%7], %8;\n\t"
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%1], [%2, {%3, %4, %5}], [%6];\n\t"
      "selp.u32 %0, 1, 0, r;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(smem_u32(next)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool tma2_load_5d_test(void* dst, const CUtensorMap* map, int x, int y, int z, int v, int w, uint32_t bar,
                                                  uint64_t* next, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred r;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 r, [%9], %10;\n\t"
      "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%1], [%2, {%3, %4, %5, %6, %7}], [%8];\n\t"
      "selp.u32 %0, 1, 0, r;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(v), "r"(w), "r"(bar), "r"(smem_u32(next)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Whole-warp operations, by one warp of each CTA of the pair.
__device__ __forceinline__ void tmem2_alloc(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem2_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem2_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// Arrive once on the barrier at `bar`'s offset in both CTAs when every MMA issued so far is done.
__device__ __forceinline__ void umma2_commit_both(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// D[tmem of both CTAs] (+)= A B^T, bf16 operands, fp32 accumulation: rows 0-127 of A and the first
// half of B's rows in the leader's shared memory, the rest at the same offsets in the peer's.  Four steps
// of 16 channels over 64, operands in 128-byte rows, by one thread of the leader, and the commit of them
// on the barrier at `done`'s offset in both CTAs.  Returns whether the phase of `next` is complete; it is
// asked for ahead of the MMAs and looked at behind them (the answer takes 180 clocks, issuing them
// 340).
__device__ __forceinline__ bool umma2_f16_step(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate, uint64_t* done, uint64_t* next, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, r, t;\n\t.reg .b64 a, b;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 r, [%8], %9;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.eq.b32 t, 0, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%1], %2, %3, %4, p;\n\t"
      "add.s64 a, %2, 2;\n\tadd.s64 b, %3, 2;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%1], a, b, %4, t;\n\t"
      "add.s64 a, %2, 4;\n\tadd.s64 b, %3, 4;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%1], a, b, %4, t;\n\t"
      "add.s64 a, %2, 6;\n\tadd.s64 b, %3, 6;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%1], a, b, %4, t;\n\t"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%6], %7;\n\t"
      "selp.u32 %0, 1, 0, r;\n\t}"
      : "=r"(ok)
      : "r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(smem_u32(done)), "h"((uint16_t)3),
        "r"(smem_u32(next)), "r"(parity)
      : "memory");
  return ok != 0;
}

}  // namespace tc
}  // namespace dsv4
