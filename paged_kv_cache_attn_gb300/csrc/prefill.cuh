// Helpers shared by the prefill kernels (latent prefill, chunk attention).
#pragma once

#include "cluster.cuh"

namespace pkv {
namespace tc {

// After a time-out loads may be in flight (else a product has waited for every
// one): about two milliseconds for them to land.
__device__ __forceinline__ void wait_for_copies() {
  const long long t0 = clock64();
  while (clock64() - t0 < (1 << 22)) {
  }
}

// Two fp32 in one operation.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 32 rows x 64 bytes of a warp (lane = row, w = its 16 words) out to dst(row)
// through 2 KB of shared memory, 16-byte pieces swizzled by the row: a store
// covers whole sectors of eight rows.
template <typename Dst>
__device__ __forceinline__ void put_rows(uint8_t* turn, const uint32_t (&w)[16],
                                         int lane, Dst dst) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(turn + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) =
        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int rr = k * 8 + (lane >> 2), c = lane & 3;
    const uint4 x = *reinterpret_cast<const uint4*>(
        turn + rr * 64 + ((c ^ ((rr >> 1) & 3)) << 4));
    if (uint8_t* d = dst(rr)) *reinterpret_cast<uint4*>(d + c * 16) = x;
  }
  __syncwarp();
}

}  // namespace tc
}  // namespace pkv
