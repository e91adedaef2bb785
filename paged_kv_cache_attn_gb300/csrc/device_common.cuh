// Device-side helpers shared by the decode kernels: mbarriers, TMA, ldmatrix,
// mma.sync, ex2, the device status word.  Inline PTX for sm_103a.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"

namespace pkv {

// A bounded wait gives up after about a second of SM clocks.
constexpr long long kWaitCycles = 1LL << 31;

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void record_status(DeviceStatus* st, uint32_t code,
                                              int detail) {
  if (atomicCAS(&st->code, 0u, code) == 0u) atomicExch(&st->detail, detail);
  atomicAdd(&st->count, 1u);
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count)
               : "memory");
}

__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(
                   bar),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Wait for the phase with the given parity to complete; false once `limit`
// SM clock cycles have passed without it.
__device__ __forceinline__ bool mbar_wait_for(uint32_t bar, uint32_t parity,
                                              long long limit) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > limit) return false;
  }
  return true;
}

__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
  return mbar_wait_for(bar, parity, kWaitCycles);
}

__device__ __forceinline__ void tma_prefetch_desc(const CUtensorMap* tm) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(tm) : "memory");
}

// 2-D tiled TMA load of one box into shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* tm,
                                            int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(tm), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// 1-D bulk copy global -> shared, completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src,
                                          uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

__device__ __forceinline__ float2 lds64f(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];"
               : "=f"(v.x), "=f"(v.y)
               : "r"(addr));
  return v;
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t& r0,
                                        uint32_t& r1, uint32_t& r2,
                                        uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t& r0,
                                          uint32_t& r1, uint32_t& r2,
                                          uint32_t& r3) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
      : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
      : "r"(addr));
}

// D = A(16x16 bf16, row) * B(16x8 bf16, col) + D, fp32 accumulate.
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4],
                                          uint32_t b0, uint32_t b1) {
  // Not volatile: no side effects, so the compiler may move it around the
  // (volatile) shared-memory loads and overlap their latency.
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 2^x with the hardware approximation (ex2.approx.ftz): 2^-inf = +0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ void st_shared_zero16(uint32_t addr) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(addr), "r"(0)
               : "memory");
}

// Arguments shared by the attention kernels (one launch, one layer).
struct SplitParams {
  const __nv_bfloat16* q;
  const int32_t* tables;
  const int32_t* seq_lens;
  const WorkItem* items;
  float2* ml;
  float* o;
  DeviceStatus* status;
  int nb, Hq, Hkv, G, max_blocks;
  int64_t num_blocks;
  int64_t partial_rows;
  float scale_log2;
  // Fused append (paged_decode_append_attn): this layer's K/V of each
  // branch's newest token, [nb][Hkv][d], and the pools they are written to;
  // all null for a plain decode step.
  const uint4* k_step;
  const uint4* v_step;
  uint4* k_pool;
  uint4* v_pool;
  // Not null: every item has all keys of its rows and writes their results here
  // ([nb][Hq][d], one kv-head); else partial rows.
  __nv_bfloat16* out;
};

// A work item read from the (caller-uploaded) plan must stay inside the
// arrays it indexes; a malformed one is recorded and skipped.
__device__ __forceinline__ bool item_ok(const WorkItem& it,
                                        const SplitParams& p, int max_rows) {
  const int64_t last_row = (int64_t)it.row0 + it.nrows - 1;
  return it.nrows >= 1 && it.nrows <= max_rows && it.row0 >= 0 &&
         it.branch0 >= 0 && it.branch0 + last_row / p.G < p.nb &&
         it.g >= 0 && it.g < p.Hkv && it.blk_begin >= 0 &&
         it.blk_begin < it.blk_end && it.blk_end <= p.max_blocks &&
         it.prow_base >= 0 &&
         (int64_t)it.prow_base + it.nrows <= p.partial_rows;
}

// Where an item's row goes in p.out.
__device__ __forceinline__ int64_t result_row(const SplitParams& p, const WorkItem& it,
                                              int row) {
  return (int64_t)it.branch0 * p.Hq + it.row0 + row;
}

// The results of a warp's own item: lane (gq, tq) has of rows gq and gq + 8 (hr) the
// columns 8 nt + 2 tq and + 1, value(nt, hr), and the rows' sums.
template <int D, typename Value>
__device__ __forceinline__ void put_results(const SplitParams& p, const WorkItem& it,
                                            int lane, float l0, float l1, Value value) {
  const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
  for (int hr = 0; hr < 2; ++hr) {
    if (gq + 8 * hr >= it.nrows) continue;
    const float inv = 1.f / (hr ? l1 : l0);
    __nv_bfloat16* dst = p.out + result_row(p, it, gq + 8 * hr) * D + 2 * tq;
#pragma unroll
    for (int nt = 0; nt < D / 8; ++nt) {
      const float2 v = value(nt, hr);
      *reinterpret_cast<uint32_t*>(dst + 8 * nt) = pack_bf16(v.x * inv, v.y * inv);
    }
  }
}

}  // namespace pkv
