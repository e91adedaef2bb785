// Cluster helpers of the latent kernels: a pair of CTAs on two SMs that hand
// tiles to each other through distributed shared memory.  Inline PTX for sm_103a.
#pragma once

#include "tcgen05.cuh"

namespace pkv {
namespace tc {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Every thread of both CTAs; ordinary memory operations before it are visible
// to both CTAs after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Address of the same shared-memory place in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(r)
               : "r"(addr), "r"(rank));
  return r;
}

// Arrive on an mbarrier of another CTA of the cluster.  Relaxed: it reports
// only that something has happened that the other side may now overwrite or
// refill (asynchronous copies and MMAs carry their own ordering).
__device__ __forceinline__ void remote_arrive(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                   cluster_bar)
               : "memory");
}

// Store into another CTA's shared memory, counted (16 or 4 bytes) on a barrier
// there.  The stores of a warp run at the full rate of the SM-to-SM network
// (21 bytes a cycle, measured) when they cover whole 128-byte lines, at half of
// it as scattered 16-byte pieces.  They are ordinary (generic proxy) writes: the
// side that feeds them to an MMA puts a proxy fence between its wait and the MMA.
__device__ __forceinline__ void remote_store16(uint32_t dst, uint32_t a,
                                               uint32_t b, uint32_t c,
                                               uint32_t d, uint32_t bar) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 "
      "[%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
      "r"(a), "r"(b), "r"(c), "r"(d), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void remote_store4(uint32_t dst, uint32_t a,
                                              uint32_t bar) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 "
      "[%0], %1, [%2];" ::"r"(dst),
      "r"(a), "r"(bar)
      : "memory");
}

// Wait with acquire at cluster scope: what another CTA sent is visible.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar,
                                                      uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar,
                                                  uint32_t parity) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait_cluster(bar, parity)) {
    if (clock64() - t0 > kWaitCycles) return false;
  }
  return true;
}

// One lane of a converged warp, the same every time.  A warp that issues MMAs
// keeps its control flow uniform and lets this lane issue: descriptors and
// addresses then stay in uniform registers (an MMA of 65 cycles took 92 to issue
// from a one-lane branch, 70 this way).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ int uniform(int v) {
  return __shfl_sync(0xffffffffu, v, 0);
}

// Warp-wide waits polled by every lane.  Polled by one lane with the others
// waiting for it, a completed barrier was seen some 700 cycles late.
__device__ __forceinline__ bool all_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

__device__ __forceinline__ bool all_wait_cluster(uint32_t bar,
                                                 uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity));
}

// Report all of this thread's earlier MMAs on the barrier at the same place
// in the CTAs of `mask`.
__device__ __forceinline__ void umma_commit_to(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster"
      ".multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}

// ---- a pair of CTAs as one unit of the tensor cores (cta_group::2) ---------------
// D of 256 rows: the even CTA's tensor memory holds rows 0-127, the odd one's rows
// 128-255, each from its own A; each CTA holds half of B's N.  One thread of the
// even CTA issues for both; addresses and descriptors hold in both CTAs.

__device__ __forceinline__ void tmem_alloc2(uint32_t where, uint32_t cols) {
  asm volatile(
      "tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
          where),
      "r"(cols)
      : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" :::
                   "memory");
}

__device__ __forceinline__ void tmem_free2(uint32_t tmem, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
               "r"(cols)
               : "memory");
}

__device__ __forceinline__ void umma2_ts(uint32_t tmem_d, uint32_t tmem_a,
                                         uint64_t b, uint32_t id,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(
          tmem_d),
      "r"(tmem_a), "l"(b), "r"(id), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void umma2_ss(uint32_t tmem_d, uint64_t a, uint64_t b,
                                         uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(
          tmem_d),
      "l"(a), "l"(b), "r"(id), "r"(accumulate)
      : "memory");
}

// Report all of this thread's earlier pair MMAs on the barrier at the same
// place in both CTAs.
__device__ __forceinline__ void umma2_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
      ".multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

// Loads of a CTA of the pair that complete on a barrier (cluster address) of
// either CTA.
__device__ __forceinline__ void tma2_load_2d(uint32_t dst, const CUtensorMap* tm,
                                             int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::"
      "bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(tm), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma2_load_3d(uint32_t dst, const CUtensorMap* tm,
                                             int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::"
      "bytes.cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(tm), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma2_load_5d_at(uint32_t dst,
                                                const CUtensorMap* tm, int x2,
                                                int x4, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::"
      "bytes.cta_group::2 [%0], [%1, {%2, %2, %3, %2, %4}], [%5];" ::"r"(dst),
      "l"(tm), "r"(0), "r"(x2), "r"(x4), "r"(bar)
      : "memory");
}

// Arrive on a barrier of a CTA of the cluster with bytes to expect there;
// relaxed like remote_arrive (a release at cluster scope took 1400 cycles).
__device__ __forceinline__ void remote_expect_tx(uint32_t cluster_bar,
                                                 uint32_t bytes) {
  asm volatile(
      "mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], "
      "%1;" ::"r"(cluster_bar),
      "r"(bytes)
      : "memory");
}

__device__ __forceinline__ void cluster_store4(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// One box of a 5-D map whose x0, x1 and x3 start at 0.
__device__ __forceinline__ void tma_load_5d_at(uint32_t dst,
                                               const CUtensorMap* tm, int x2,
                                               int x4, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%2, %2, %3, %2, %4}], [%5];" ::"r"(dst),
      "l"(tm), "r"(0), "r"(x2), "r"(x4), "r"(bar)
      : "memory");
}

// 128 rows x 32 bytes from shared memory (the layout of a K-major operand,
// descriptor as for an MMA) to 8 columns of tensor memory; runs in order with
// the thread's later MMAs.
__device__ __forceinline__ void umma_copy(uint32_t tmem_d, uint64_t src) {
  asm volatile("tcgen05.cp.cta_group::1.128x256b [%0], %1;" ::"r"(tmem_d), "l"(src)
               : "memory");
}

// K-major operand descriptor without swizzle: 8 rows x 16 bytes are 128
// contiguous bytes, `k` bytes apart along K and `m` bytes along the rows.
__device__ __forceinline__ uint64_t sdesc_plain(uint32_t addr, uint32_t k,
                                                uint32_t m) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) |
         ((uint64_t)((k >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((m >> 4) & 0x3FFFu) << 32) | (1ull << 46);
}

// Ask for one box of a 2-D map in L2.
__device__ __forceinline__ void l2_prefetch_2d(const CUtensorMap* tm, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(tm),
               "r"(x), "r"(y)
               : "memory");
}

// Named barriers over `n` threads (whole warps), combining a predicate.
__device__ __forceinline__ bool bar_and(int id, int n, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred.aligned q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

}  // namespace tc
}  // namespace pkv
