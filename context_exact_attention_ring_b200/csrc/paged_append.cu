// New K and V rows written into the pages of a cache: row t of k_new and v_new
// [T, Hkv, D] goes to cache row slot_map[t] = page * ps + offset of the pools.
// A slot outside the pools (-1: padding, or a token that found no page) is
// skipped.
//
// A copy: bound by memory.  The call's 16-byte pieces (T rows of K and of V)
// are numbered through and dealt to the threads of blocks of 1024 pieces, four
// independent loads each before the four stores, so that a single token's row
// is spread over as many threads as it has pieces and a prompt's over the GPU
// (32k tokens of 8 x 128 bf16: 43 us, 6.2 TB/s read and written).
#include <cuda_runtime.h>

#include "paged.cuh"

namespace ra {

namespace pga {
constexpr int THREADS = 256;
constexpr int PER = 4;     // 16-byte pieces per thread
}  // namespace pga

__global__ void __launch_bounds__(pga::THREADS) paged_append_kernel(PagedAppendArgs a, int nvh, int nv) {
  using namespace pga;
  // nvh: pieces of a head's row, nv: of a token's K and V rows together (K first)
  paged_begin();
  const long long total = (long long)a.T * nv;
  const long long first = (long long)blockIdx.x * (THREADS * PER);
  const int t0 = (int)(first / nv), e0 = (int)(first - (long long)t0 * nv);
  uint4 x[PER];
  uint8_t* dst[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int o = e0 + i * THREADS + threadIdx.x;     // below nv + 1024
    const int dt = o / nv;
    int e = o - dt * nv;
    const int t = t0 + dt;
    dst[i] = nullptr;
    if (first + i * THREADS + threadIdx.x >= total) continue;
    const int slot = a.slot_map[t];
    const int page = slot >> a.ps_log2;
    if (slot < 0 || page >= a.num_pages) continue;
    const bool is_v = e >= nv / 2;
    if (is_v) e -= nv / 2;
    const int h = e / nvh, c = e - h * nvh;
    const uint8_t* src = static_cast<const uint8_t*>(is_v ? a.v_new : a.k_new) +
                         ((long long)t * a.new_token + (long long)h * a.new_head) * a.elem_bytes + c * 16;
    x[i] = *reinterpret_cast<const uint4*>(src);
    dst[i] = static_cast<uint8_t*>(is_v ? a.v_pool : a.k_pool) +
             ((long long)page * a.pool.page + (long long)(slot & ((1 << a.ps_log2) - 1)) * a.pool.token +
              (long long)h * a.pool.head) * a.elem_bytes + c * 16;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (dst[i]) *reinterpret_cast<uint4*>(dst[i]) = x[i];
}

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t st) {
  const int nvh = a.D * a.elem_bytes / 16, nv = 2 * a.Hkv * nvh;
  const long long total = (long long)a.T * nv, per = pga::THREADS * pga::PER;
  const long long blocks = (total + per - 1) / per;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return paged_launch(paged_append_kernel, (unsigned)blocks, pga::THREADS, 0, st, a, nvh, nv);
}

}  // namespace ra
