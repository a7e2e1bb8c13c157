// Block tables and slot maps of a paged KV cache, kept on the device.
//
// page_extend makes room for new tokens: sequence b of length len_b gets
//   need_b = ceil((len_b + new_b) / ps) - ceil(len_b / ps)
// pages from the end of the free list, in order of sequence and page, and the
// call's tokens, packed sequence after sequence, get their cache rows
//   slot(t) = page(pos / ps) * ps + pos % ps,   pos = len_b + t - cu_b.
// Two prefix sums over the sequences (tokens, then pages, since whether a
// sequence's tokens fit decides whether it takes pages) run in one block,
// which also moves the pages.  The slots are one independent lookup each: a few
// thousand are written by the same block (a page not in the table before the
// call is looked up in the free list, so nothing waits for the table), more by
// a second launch over the whole GPU.  Latency-bound: a decode step moves a few
// KB.
//
// page_trim shortens sequences and puts the pages past their new ends back,
// last taken on top, so that extending and trimming by the same tokens leaves
// the free list as it was.  A table entry that marks an absent page is not put
// there.
#include <cuda_runtime.h>

#include "kernels.h"
#include "paged.cuh"

namespace ra {

namespace pgt {
constexpr int THREADS = 1024;             // of the block that scans; sequences of a chunk
constexpr int NW = THREADS / 32;
constexpr int ONE_LAUNCH_TOKENS = 4096;   // slots written by the first launch's block: 4 a thread
constexpr int SLOT_THREADS = 256, SLOTS = 4;   // of the second launch: slots a thread
}  // namespace pgt

// Inclusive prefix sum over the block's threads; *total gets the sum of all.
// Ends with every thread past its reads of s_warp.
__device__ __forceinline__ long long block_scan(long long x, long long* s_warp, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += up;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  long long w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += up;
  }
  const long long before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
  *total = __shfl_sync(0xffffffffu, w, 31);
  __syncthreads();
  return warp ? x + before : x;
}

__device__ __forceinline__ int pages_of(long long len, int ps_log2) {
  return (int)((len + (1 << ps_log2) - 1) >> ps_log2);
}

// Last i in [lo, hi) with v[i] <= x (v ascending, v[lo] <= x).
template <typename T>
__device__ __forceinline__ int last_at_most(const T* v, int lo, int hi, T x) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Whether a table entry can be a page of a pool, whose slots are 32-bit numbers: an absent page is not.
__device__ __forceinline__ bool is_page(int page, int ps_log2) { return page >= 0 && page <= (0x7fffffff >> ps_log2); }

__device__ __forceinline__ int slot_at(int page, int pos, int ps_log2) {
  if (!is_page(page, ps_log2)) return -1;
  return (page << ps_log2) | (pos & ((1 << ps_log2) - 1));
}

struct ScanSmem {
  long long warp[pgt::NW];
  long long off[pgt::THREADS];    // pages moved for the chunk's sequences before this one
  int from[pgt::THREADS];         // first page of the table it concerns
  int count[pgt::THREADS];        // pages moved
  int cu[pgt::THREADS], start[pgt::THREADS];
  int long_seq[pgt::THREADS], n_long;
};

// Moves pages j < s.count[i] of the chunk's n sequences: store(i, j, load(i, j)).
// `total` pages are numbered through in s.off (those of a sequence that is not
// served among them).  Up to four a thread, a thread finds its pages' sequences
// by bisection.  More, a warp takes a sequence's first 128, four sequences'
// 64 in flight at once, and the block together the rest of the long ones.
// (Extend and trim of 256 sequences with 40 pages: 7.5 us by bisection, 10 the
// other way; of 1021 sequences with 33,000 pages: 65 and 33 us.)  Called by all
// threads between barriers.
template <typename Load, typename Store>
__device__ __forceinline__ void move_pages(ScanSmem& s, int n, long long total, Load load, Store store) {
  using namespace pgt;
  constexpr int OWN = 128;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (total <= 4 * THREADS) {
    for (long long g = tid; g < total; g += THREADS) {
      const int i = last_at_most(s.off, 0, n, g), j = (int)(g - s.off[i]);
      if (j < s.count[i]) store(i, j, load(i, j));
    }
    return;
  }
  if (tid < n && s.count[tid] > OWN) s.long_seq[atomicAdd(&s.n_long, 1)] = tid;
  for (int i0 = warp; i0 < n; i0 += 4 * NW) {
    int count[4], most = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      count[u] = i0 + u * NW < n ? min(s.count[i0 + u * NW], OWN) : 0;
      most = max(most, count[u]);
    }
    for (int j0 = lane; j0 < most + lane; j0 += 64) {       // the same number of turns in every lane
      int v[4][2];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int k = 0; k < 2; ++k) v[u][k] = j0 + 32 * k < count[u] ? load(i0 + u * NW, j0 + 32 * k) : 0;
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (j0 + 32 * k < count[u]) store(i0 + u * NW, j0 + 32 * k, v[u][k]);
    }
  }
  __syncthreads();
  for (int q = 0; q < s.n_long; ++q) {
    const int i = s.long_seq[q], m = s.count[i];
    for (int j0 = OWN + tid; j0 < m; j0 += 4 * THREADS) {
      int v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = j0 + u * THREADS < m ? load(i, j0 + u * THREADS) : 0;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (j0 + u * THREADS < m) store(i, j0 + u * THREADS, v[u]);
    }
  }
}

// One_launch: at most THREADS sequences and ONE_LAUNCH_TOKENS slots, written here.
__global__ void __launch_bounds__(pgt::THREADS, 1) page_extend_kernel(ExtendArgs a, int one_launch) {
  using namespace pgt;
  __shared__ ScanSmem s;
  paged_begin();
  const int tid = threadIdx.x;
  const long long cap = (long long)a.W << a.ps_log2;
  const int n_free = min(max(*a.n_free, 0), a.max_free);
  long long tokens = 0, pages = 0, taken = 0;   // of the sequences before this chunk; pages this call takes
  bool full = false;
  unsigned largest = 0;       // of the pages given out: one that is no page leaves its tokens without slots
  for (int b0 = 0; b0 < a.B; b0 += THREADS) {
    const int b = b0 + tid, in_chunk = min(THREADS, a.B - b0);
    const bool in = b < a.B;
    const long long len = in ? min(max((long long)a.seq_lens[b], 0LL), cap) : 0;
    const long long add = in ? max(a.new_lens[b], 0) : 0;
    long long total;
    const long long cu1 = tokens + block_scan(add, s.warp, &total);
    const long long cu0 = cu1 - add;
    tokens += total;
    const bool fits = in && len + add <= cap && (add == 0 || cu1 <= a.max_tokens);
    const int old = pages_of(len, a.ps_log2);
    const int need = fits ? pages_of(len + add, a.ps_log2) - old : 0;
    const long long upto = block_scan(need, s.warp, &total);
    // the sequences served take the first pages of the list without a gap: once one finds too few,
    // no later one that needs any is served
    const bool ok = fits && (need == 0 || pages + upto <= n_free);
    full |= in && !ok;
    if (in) {
      if (b == 0) a.cu_new[0] = 0;
      a.cu_new[b + 1] = (int)min(cu1, 0x7fffffffLL);
      a.start_lens[b] = ok ? (int)len : -1;
      if (ok) a.seq_lens[b] = (int)(len + add);
    }
    s.off[tid] = upto - need;
    s.from[tid] = old;
    s.cu[tid] = (int)min(cu0, 0x7fffffffLL);
    s.start[tid] = ok ? (int)len : -1;
    s.count[tid] = ok ? need : 0;
    if (tid == 0) s.n_long = 0;
    const long long mine = ok && need ? pages + upto : 0;     // the last that this sequence takes
    taken = max(taken, mine);
    __syncthreads();
    move_pages(s, in_chunk, total, [&](int i, int j) { return __ldg(a.free_pages + (n_free - 1 - (pages + s.off[i] + j))); },
               [&](int i, int j, int page) {
                 a.table[(size_t)(b0 + i) * a.table_stride + s.from[i] + j] = page;
                 largest = max(largest, (unsigned)page);
               });
    if (one_launch) {
#pragma unroll 4
      for (int t = tid; t < a.max_tokens; t += THREADS) {
        int slot = -1;
        if (t < tokens) {
          const int i = last_at_most(s.cu, 0, in_chunk, t);
          if (s.start[i] >= 0) {
            const int pos = s.start[i] + (t - s.cu[i]), p = pos >> a.ps_log2;
            const int page = p < s.from[i] ? a.table[(size_t)i * a.table_stride + p]
                                           : a.free_pages[n_free - 1 - (s.off[i] + p - s.from[i])];
            slot = slot_at(page, pos, a.ps_log2);
          }
        }
        a.slot_map[t] = slot;
      }
    }
    pages += total;
    __syncthreads();    // s is free
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
  if ((tid & 31) == 0) s.warp[tid >> 5] = taken;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < NW; ++w) taken = max(taken, s.warp[w]);
    *a.n_free = n_free - (int)taken;
  }
  if ((full || !is_page((int)largest, a.ps_log2)) && a.err) atomicCAS(a.err, 0u, kFaultCapacity);
}

// Slots [first, first + SLOT_THREADS * SLOTS) by each block: a warp finds the
// sequence of the first and one that of the last (32 probes at once), the
// threads bisect between them.
__global__ void __launch_bounds__(pgt::SLOT_THREADS) slot_map_kernel(ExtendArgs a) {
  using namespace pgt;
  __shared__ int s_seq[2];
  paged_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = blockIdx.x * (SLOT_THREADS * SLOTS);
  const int last = min(first + (SLOT_THREADS * SLOTS - 1), a.max_tokens - 1);    // below 2^31 whatever max_tokens
  const int all = a.cu_new[a.B];
  if (warp < 2) {
    const int t = min(warp ? last : first, max(all - 1, 0));
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, at = lo + lane * step;
      const uint32_t le = __ballot_sync(0xffffffffu, at < hi && a.cu_new[min(at, a.B)] <= t);
      lo += (__popc(le) - 1) * step;      // lane 0 always agrees
      hi = min(hi, lo + step);
    }
    if (lane == 0) s_seq[warp] = lo;
  }
  __syncthreads();
  const int lo = s_seq[0], hi = s_seq[1] + 1;
#pragma unroll
  for (int u = 0; u < SLOTS; ++u) {
    const int t = first + u * SLOT_THREADS + threadIdx.x;
    if (t > last) break;
    int slot = -1;
    if (t < all) {
      const int b = last_at_most(a.cu_new, lo, hi, t);
      const int start = a.start_lens[b];
      if (start >= 0) {
        const int pos = start + (t - a.cu_new[b]);
        slot = slot_at(a.table[(size_t)b * a.table_stride + (pos >> a.ps_log2)], pos, a.ps_log2);
      }
    }
    a.slot_map[t] = slot;
  }
}

cudaError_t launch_page_extend(const ExtendArgs& a, cudaStream_t st) {
  const int one = a.max_tokens <= pgt::ONE_LAUNCH_TOKENS && a.B <= pgt::THREADS;
  const cudaError_t e = paged_launch(page_extend_kernel, 1, pgt::THREADS, 0, st, a, one);
  if (e != cudaSuccess || one) return e;
  constexpr int per = pgt::SLOT_THREADS * pgt::SLOTS;
  return paged_launch(slot_map_kernel, (a.max_tokens - 1) / per + 1, pgt::SLOT_THREADS, 0, st, a);
}

// Puts the chunk's pages (n sequences, `total` table entries numbered through
// in s.off) onto the list from `base` up, the last one first, without the
// entries that are no page.  Returns how many pages there are.
__device__ __forceinline__ long long trim_present(const TrimArgs& a, ScanSmem& s, int b0, int n, long long total,
                                               long long base) {
  using namespace pgt;
  long long done = 0;
  for (long long g0 = 0; g0 < total; g0 += THREADS) {
    const long long g = total - 1 - g0 - threadIdx.x;
    int page = -1;
    if (g >= 0) {
      const int i = last_at_most(s.off, 0, n, g);
      page = a.table[(size_t)(b0 + i) * a.table_stride + s.from[i] + (g - s.off[i])];
    }
    const bool present = is_page(page, a.ps_log2);
    long long turn;
    const long long to = base + done + block_scan(present, s.warp, &turn) - 1;
    if (present && to < a.max_free) a.free_pages[to] = page;
    done += turn;
  }
  return done;
}

// The last chunk of sequences first: its pages lie lowest on the list.
__global__ void __launch_bounds__(pgt::THREADS, 1) page_trim_kernel(TrimArgs a) {
  using namespace pgt;
  __shared__ ScanSmem s;
  paged_begin();
  const int tid = threadIdx.x;
  const long long cap = (long long)a.W << a.ps_log2;
  long long base = min(max(*a.n_free, 0), a.max_free), total;
  for (int b0 = (a.B - 1) / THREADS * THREADS; b0 >= 0; b0 -= THREADS) {
    const int b = b0 + tid, in_chunk = min(THREADS, a.B - b0);
    long long len = 0, keep = 0;
    if (b < a.B) {
      len = min(max((long long)a.seq_lens[b], 0LL), cap);
      keep = min(max((long long)a.keep_lens[b], 0LL), len);
    }
    const int from = pages_of(keep, a.ps_log2);
    const int gone = pages_of(len, a.ps_log2) - from;
    const long long upto = block_scan(gone, s.warp, &total);
    s.off[tid] = upto - gone;
    s.from[tid] = from;
    s.count[tid] = gone;
    if (tid == 0) s.n_long = 0;
    if (b < a.B) a.seq_lens[b] = (int)keep;
    __syncthreads();
    // as if every entry were a page; where one is not (rare), the chunk's pages are placed again
    unsigned largest = 0;
    move_pages(s, in_chunk, total,
               [&](int i, int j) { return __ldg(a.table + (size_t)(b0 + i) * a.table_stride + s.from[i] + j); },
               [&](int i, int j, int page) {
                 const long long to = base + total - 1 - (s.off[i] + j);
                 if (to < a.max_free) a.free_pages[to] = page;     // the list cannot hold more
                 largest = max(largest, (unsigned)page);
               });
    if (__syncthreads_or(!is_page((int)largest, a.ps_log2))) {
      total = trim_present(a, s, b0, in_chunk, total, base);
      __syncthreads();
    }
    base += total;      // s is free
  }
  if (tid == 0) {
    *a.n_free = (int)min(base, (long long)a.max_free);
    if (base > a.max_free && a.err) atomicCAS(a.err, 0u, kFaultCapacity);
  }
}

cudaError_t launch_page_trim(const TrimArgs& a, cudaStream_t st) {
  return paged_launch(page_trim_kernel, 1, pgt::THREADS, 0, st, a);
}

}  // namespace ra
