// What the operators around the layer share about shared memory: the opt-in above 48 KB
// and the copy of a whole row (one instruction, counted on an mbarrier).
#pragma once

#include <mutex>

#include "tma.cuh"

namespace moe {
namespace {

// The kernel's shared-memory opt-in, once per device.
template <typename Kernel>
bool opt_in(Kernel kern, int bytes, std::mutex& mu, bool (&done)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  std::lock_guard<std::mutex> lock(mu);
  if (!done[dev]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
        cudaSuccess)
      return false;
    done[dev] = true;
  }
  return true;
}

// `bytes` (a multiple of 16, both addresses too) from global to shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

}  // namespace
}  // namespace moe
