// Per-kernel host set-up of the 16/32-bit operators, done once per device: the dynamic
// shared-memory limit and the number of resident blocks per SM. Both are properties of
// the kernel alone; asking for them on every call costs more than the launch.
#pragma once

#include <atomic>

#include "common.cuh"

namespace lnfp8 {

template <auto Kernel>
lnfp8_status kernel_setup(int threads, size_t smem, int* blocks_per_sm, const char* who) {
  static std::atomic<int> known[64];  // resident blocks + 1; 0: not asked yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return check_launch(who);
  std::atomic<int>* slot = dev >= 0 && dev < 64 ? &known[dev] : nullptr;
  int n = slot ? slot->load(std::memory_order_relaxed) - 1 : -1;
  if (n < 0) {
    if (smem > 0 && cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
      return check_launch(who);
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, Kernel, threads, smem) != cudaSuccess) return check_launch(who);
    if (n < 1) n = 1;
    if (slot) slot->store(n + 1, std::memory_order_relaxed);
  }
  if (blocks_per_sm) *blocks_per_sm = n;
  return LNFP8_OK;
}

}  // namespace lnfp8
