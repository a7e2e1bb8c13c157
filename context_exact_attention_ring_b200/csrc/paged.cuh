// Device helpers the paged-cache kernels share.
#pragma once
#include "paged.h"
#include "ptx.cuh"

namespace ra {

// All threads, before the first access to global memory: lets the next kernel
// of the stream start early, and waits until the one before has completed.
// No thread skips the wait, so a kernel's completion implies that of all
// kernels before it on the stream.
__device__ __forceinline__ void paged_begin() {
  grid_launch_dependents();
  grid_dependency_wait();
}

// Maximum over the warp's lanes (NaN ignored, as fmaxf does).
__device__ __forceinline__ float warp_max_redux(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

}  // namespace ra
