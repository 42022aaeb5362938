// smem.cuh -- kernels with more dynamic shared memory than the default limit.
#pragma once
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

namespace nvfp4 {

// The most dynamic shared memory that a kernel is ever launched with, asked for
// once per device (`done`: one word per kernel).  The limit belongs to the
// kernel, not to a launch: a call that set its own size would take away what
// another host thread's launch needs.
template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && done.load(std::memory_order_relaxed) >> dev & 1)) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess && dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  return e;
}

}  // namespace nvfp4
