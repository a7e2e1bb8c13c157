// Device helpers the paged-cache kernels share.
#pragma once
#include "paged.h"
#include "ptx.cuh"

namespace ra {

// All threads, before the first access to global memory: waits until the
// kernel before it on the stream has completed.  No thread skips the wait, so a
// kernel's completion implies that of all kernels before it.  The next kernel
// is not invited in early (griddepcontrol.launch_dependents): a ring step may
// follow, which reads its shards and blocks without waiting, and these may be
// what the kernel here writes.  It starts as this one's CTAs exit.
__device__ __forceinline__ void paged_begin() { grid_dependency_wait(); }

// Maximum over the warp's lanes (NaN ignored, as fmaxf does).
__device__ __forceinline__ float warp_max_redux(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

}  // namespace ra
