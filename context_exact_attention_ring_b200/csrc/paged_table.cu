// Block tables and slot maps of a paged KV cache, kept on the device.
//
// page_extend makes room for new tokens: sequence b of length len_b gets
//   need_b = ceil((len_b + new_b) / ps) - ceil(len_b / ps)
// pages from the end of the free list, in order of sequence and page, and the
// call's tokens, packed sequence after sequence, get their cache rows
//   slot(t) = table[b][pos / ps] * ps + pos % ps,   pos = len_b + t - cu_b.
// Two prefix sums over the sequences (tokens, then pages, since whether a
// sequence's tokens fit decides whether it takes pages) run in one block, which
// also moves the pages.  The slots are one independent lookup each: a few
// thousand are written by the same block, more by a second launch over the
// whole GPU.
//
// page_trim shortens sequences and puts the pages past their new ends back,
// last taken on top, so that extending and trimming by the same tokens leaves
// the free list as it was.
#include <cuda_runtime.h>

#include "kernels.h"
#include "paged.cuh"

namespace ra {

namespace pgt {
constexpr int THREADS = 1024;
constexpr int NW = THREADS / 32;
constexpr int ONE_LAUNCH_TOKENS = 4096;   // slots written by the first launch's block
}  // namespace pgt

// Inclusive prefix sum over the block's threads; *total gets the sum of all.
__device__ __forceinline__ long long block_scan(long long x, long long* s_warp, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += up;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    long long w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += up;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  if (warp > 0) x += s_warp[warp - 1];
  *total = s_warp[pgt::NW - 1];
  __syncthreads();
  return x;
}

__device__ __forceinline__ int pages_of(long long len, int ps_log2) {
  return (int)((len + (1 << ps_log2) - 1) >> ps_log2);
}

// The slot of token t.
__device__ __forceinline__ int slot_of(const ExtendArgs& a, int t) {
  // last b with cu[b] <= t
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu_new[mid] <= t) lo = mid; else hi = mid;
  }
  if (t >= a.cu_new[a.B]) return -1;
  const int start = a.start_lens[lo];
  if (start < 0) return -1;
  const int pos = start + (t - a.cu_new[lo]);
  const int page = a.table[(size_t)lo * a.table_stride + (pos >> a.ps_log2)];
  if (page < 0 || page > (0x7fffffff >> a.ps_log2)) return -1;
  return (page << a.ps_log2) | (pos & ((1 << a.ps_log2) - 1));
}

__global__ void __launch_bounds__(pgt::THREADS, 1) page_extend_kernel(ExtendArgs a, int with_slots) {
  using namespace pgt;
  __shared__ long long s_warp[NW];
  __shared__ int s_old[THREADS], s_need[THREADS];
  __shared__ long long s_off[THREADS];
  paged_begin();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long cap = (long long)a.W << a.ps_log2;
  const int n_free = min(max(*a.n_free, 0), a.max_free);
  long long tokens = 0, pages = 0, taken = 0;   // of the sequences before this chunk
  bool full = false;
  for (int b0 = 0; b0 < a.B; b0 += THREADS) {
    const int b = b0 + tid;
    const bool in = b < a.B;
    const long long len = in ? min(max((long long)a.seq_lens[b], 0LL), cap) : 0;
    const long long add = in ? max(a.new_lens[b], 0) : 0;
    long long total;
    const long long cu1 = tokens + block_scan(add, s_warp, &total);
    tokens += total;
    const bool fits = in && len + add <= cap && cu1 <= a.max_tokens;
    const int old = pages_of(len, a.ps_log2);
    const int need = fits ? pages_of(len + add, a.ps_log2) - old : 0;
    const long long upto = pages + block_scan(need, s_warp, &total);
    pages += total;
    const bool ok = fits && (need == 0 || upto <= n_free);
    full |= in && !ok;
    const long long got = block_scan(ok ? need : 0, s_warp, &total);
    (void)got;
    taken += total;
    if (in) {
      if (b == 0) a.cu_new[0] = 0;
      a.cu_new[b + 1] = (int)min(cu1, 0x7fffffffLL);
      a.start_lens[b] = ok ? (int)len : -1;
      if (ok) a.seq_lens[b] = (int)(len + add);
    }
    s_old[tid] = old;
    s_need[tid] = ok ? need : 0;
    s_off[tid] = upto - need;
    __syncthreads();
    // a warp per sequence moves its pages
    for (int i = warp; i < THREADS && b0 + i < a.B; i += NW)
      for (int j = lane; j < s_need[i]; j += 32)
        a.table[(size_t)(b0 + i) * a.table_stride + s_old[i] + j] = a.free_pages[n_free - 1 - (s_off[i] + j)];
    __syncthreads();
  }
  if (tid == 0) *a.n_free = n_free - (int)taken;
  if (full) atomicCAS(a.err, 0u, kFaultCapacity);
  if (with_slots)
    for (int t = tid; t < a.max_tokens; t += THREADS) a.slot_map[t] = slot_of(a, t);
}

__global__ void __launch_bounds__(256) slot_map_kernel(ExtendArgs a) {
  paged_begin();
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t < a.max_tokens) a.slot_map[t] = slot_of(a, t);
}

cudaError_t launch_page_extend(const ExtendArgs& a, cudaStream_t st) {
  const int one = a.max_tokens <= pgt::ONE_LAUNCH_TOKENS;
  const cudaError_t e = paged_launch(page_extend_kernel, 1, pgt::THREADS, 0, st, a, one);
  if (e != cudaSuccess || one) return e;
  return paged_launch(slot_map_kernel, (a.max_tokens + 255) / 256, 256, 0, st, a);
}

__global__ void __launch_bounds__(pgt::THREADS, 1) page_trim_kernel(TrimArgs a) {
  using namespace pgt;
  __shared__ long long s_warp[NW];
  __shared__ int s_from[THREADS], s_gone[THREADS];
  __shared__ long long s_off[THREADS];
  paged_begin();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long cap = (long long)a.W << a.ps_log2;
  const int n_free = min(max(*a.n_free, 0), a.max_free);
  // pages given back by all sequences
  long long all = 0;
  for (int b = tid; b < a.B; b += THREADS) {
    const long long len = min(max((long long)a.seq_lens[b], 0LL), cap);
    const long long keep = min(max((long long)a.keep_lens[b], 0LL), len);
    all += pages_of(len, a.ps_log2) - pages_of(keep, a.ps_log2);
  }
  long long total;
  block_scan(all, s_warp, &total);
  all = total;
  const long long room = min(all, (long long)a.max_free - n_free);   // the list cannot hold more
  long long before = 0;
  for (int b0 = 0; b0 < a.B; b0 += THREADS) {
    const int b = b0 + tid;
    long long len = 0, keep = 0;
    if (b < a.B) {
      len = min(max((long long)a.seq_lens[b], 0LL), cap);
      keep = min(max((long long)a.keep_lens[b], 0LL), len);
    }
    const int from = pages_of(keep, a.ps_log2);
    const int gone = pages_of(len, a.ps_log2) - from;
    const long long upto = before + block_scan(gone, s_warp, &total);
    before += total;
    s_from[tid] = from;
    s_gone[tid] = gone;
    s_off[tid] = upto - gone;
    __syncthreads();
    for (int i = warp; i < THREADS && b0 + i < a.B; i += NW)
      for (int j = lane; j < s_gone[i]; j += 32) {
        const long long to = n_free + all - 1 - (s_off[i] + j);
        if (to < a.max_free) a.free_pages[to] = a.table[(size_t)(b0 + i) * a.table_stride + s_from[i] + j];
      }
    if (b < a.B) a.seq_lens[b] = (int)keep;
    __syncthreads();
  }
  if (tid == 0) {
    *a.n_free = n_free + (int)room;
    if (room < all) atomicCAS(a.err, 0u, kFaultCapacity);
  }
}

cudaError_t launch_page_trim(const TrimArgs& a, cudaStream_t st) {
  return paged_launch(page_trim_kernel, 1, pgt::THREADS, 0, st, a);
}

}  // namespace ra
