// 64-bit loads from another CTA's shared memory, for the kernels whose clusters
// exchange fp64 sums or 64-bit keys, sm_100a.
#pragma once
#include <cstdint>

namespace fn {

__device__ __forceinline__ unsigned long long dsmem_ld_u64(uint32_t addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

}  // namespace fn
