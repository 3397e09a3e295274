// PTX wrappers that the prompt and eviction kernels need beside ptx.cuh.
#pragma once

#include "ptx.cuh"

namespace mlra {
namespace ptx {

// Waits (bounded, whether or not the CTA has given up) for work of this CTA
// that is still in flight, before a kernel that gave up leaves.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > kWaitCycles / 100) return;
}

// A barrier among `threads` threads of the CTA (whole warps).
__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

}  // namespace ptx
}  // namespace mlra
