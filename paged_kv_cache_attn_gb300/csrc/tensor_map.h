// Host helpers shared by the kernels' launchers: tensor maps and the
// shared-memory opt-in.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "internal.h"

namespace pkv {

// A tiled map over bf16 data with 128-byte swizzle and zero fill (decode.cu).
// strides: bytes, rank - 1 of them.
kv_status encode_bf16_map(CUtensorMap* tm, const void* base, int rank,
                          const cuuint64_t* dims, const cuuint64_t* strides,
                          const cuuint32_t* box);

// Allow `kernel` `bytes` of dynamic shared memory on the current device, once
// per device (`done`: a bit per device, one word per kernel).
template <typename Kernel>
cudaError_t opt_in_smem(Kernel kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Launch a kernel that may start before the one ahead of it in the stream has
// ended (it waits for that by griddepcontrol.wait).
template <typename... Formal, typename... Args>
cudaError_t launch_early(void (*kernel)(Formal...), int grid, int block, int smem,
                         cudaStream_t st, const Args&... args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace pkv
