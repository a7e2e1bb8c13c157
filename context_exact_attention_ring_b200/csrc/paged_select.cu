// Which pages of a long cache a query needs: bounds, scores, selection.
//
// bounds   per page and kv head the elementwise minimum lo and maximum hi of
//          the page's valid keys (comparisons only: exact in the cache's type).
// scores   score(page) = max over the heads h of the group of
//            sum_d max(q_hd lo_d, q_hd hi_d) >= max_h max_{key in page} q_h . k,
//          so no key of a page scores above it but by the rounding of float32 sums.
// select   the K best pages of a (sequence, kv head), in ascending order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "kernels.h"
#include "paged.cuh"

namespace ra {

// ---------------------------------------------------------------------------
// bounds.  Bound by the bytes of the keys: a thread takes a 16-byte column of
// a page's rows (all heads of a token are neighbours in the usual layout, so
// a page is read in whole lines), 8 rows in flight.  The columns of all pages
// of a sequence are numbered through, so that pages of few heads fill blocks
// as well.  bf16 pairs are compared two at a time.  (1.07 GB of keys in 171 us,
// 6.7 TB/s with the bounds written.)
// ---------------------------------------------------------------------------
namespace pgb {
constexpr int THREADS = 256;
}

// four 32-bit words of float or of two bf16 each: minimum / maximum that keep a NaN
template <typename T>
struct Word;
template <>
struct Word<float> {
  static constexpr uint32_t MAX = 0x7f800000u, MIN = 0xff800000u;   // +inf, -inf
  __device__ __forceinline__ static uint32_t lo(uint32_t a, uint32_t b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
    return __float_as_uint(r);
  }
  __device__ __forceinline__ static uint32_t hi(uint32_t a, uint32_t b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
    return __float_as_uint(r);
  }
};
template <>
struct Word<__nv_bfloat16> {
  static constexpr uint32_t MAX = 0x7f807f80u, MIN = 0xff80ff80u;
  __device__ __forceinline__ static uint32_t lo(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ __forceinline__ static uint32_t hi(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};

template <typename T>
__global__ void __launch_bounds__(pgb::THREADS) page_bounds_kernel(BoundsArgs a) {
  paged_begin();
  constexpr int E = 16 / sizeof(T);      // elements of a column
  constexpr int U = 8;                   // rows in flight (pages hold at least 8)
  const int b = blockIdx.y, ps = 1 << a.ps_log2;
  const int len = min(max(a.seq_lens[b], 0), a.W << a.ps_log2);
  const int start = a.start_lens ? a.start_lens[b] : 0;
  if (start < 0) return;      // no new tokens
  const int p0 = start >> a.ps_log2;
  const int np = (len + ps - 1) >> a.ps_log2;
  const int nc = a.Hkv * a.D / E, step = gridDim.x * pgb::THREADS;
  const int dp = step / nc, dc = step - dp * nc;
  int p = p0 + (blockIdx.x * pgb::THREADS + threadIdx.x) / nc;
  int c = (blockIdx.x * pgb::THREADS + threadIdx.x) % nc;
  for (; p < np; p += dp, c += dc) {
    if (c >= nc) {
      c -= nc;
      if (++p >= np) break;
    }
    const int page = a.table[(size_t)b * a.table_stride + p];
    if (page < 0 || page >= a.num_pages) continue;
    const int rows = min(ps, len - (p << a.ps_log2));
    const int h = c * E / a.D, d = c * E - h * a.D;
    const T* k = static_cast<const T*>(a.k) + (long long)page * a.pool.page + (long long)h * a.pool.head + d;
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = Word<T>::MAX;
      hi[i] = Word<T>::MIN;
    }
    auto take = [&](const uint4& x) {
      lo[0] = Word<T>::lo(lo[0], x.x); hi[0] = Word<T>::hi(hi[0], x.x);
      lo[1] = Word<T>::lo(lo[1], x.y); hi[1] = Word<T>::hi(hi[1], x.y);
      lo[2] = Word<T>::lo(lo[2], x.z); hi[2] = Word<T>::hi(hi[2], x.z);
      lo[3] = Word<T>::lo(lo[3], x.w); hi[3] = Word<T>::hi(hi[3], x.w);
    };
    for (int r = 0; r < rows; r += U) {
      // past the last valid row that row again: it changes nothing
      uint4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        x[u] = *reinterpret_cast<const uint4*>(k + (long long)min(r + u, rows - 1) * a.pool.token);
#pragma unroll
      for (int u = 0; u < U; ++u) take(x[u]);
    }
    T* o = static_cast<T*>(a.bounds) + ((long long)page * a.Hkv + h) * 2 * a.D + d;
    *reinterpret_cast<uint4*>(o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4*>(o + a.D) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
}

cudaError_t launch_page_bounds(const BoundsArgs& a, cudaStream_t st) {
  // enough blocks to fill the GPU, no more than a sequence's table has columns
  const long long cols = (long long)a.W * (a.Hkv * a.D * a.elem_bytes / 16);
  const long long most = (cols + pgb::THREADS - 1) / pgb::THREADS;
  const int fill = max(1, num_sms() * 16 / a.B);
  const dim3 grid((unsigned)(most < fill ? most : fill), a.B);
  if (a.elem_bytes == 2) return paged_launch(page_bounds_kernel<__nv_bfloat16>, grid, pgb::THREADS, 0, st, a);
  return paged_launch(page_bounds_kernel<float>, grid, pgb::THREADS, 0, st, a);
}

// ---------------------------------------------------------------------------
// scores.  Bound by the bytes of the bounds.  A half-warp shares a page, 8 (or
// 4) dims a lane in 16-byte pieces, and holds two pages at once; the group's
// queries wait in shared memory, so that any number of heads takes one pass.
// max(q lo, q hi) is q times hi or lo by the sign of q: a select and an FMA.
// The two pages' sums are added up across the half-warp by halving: after one
// exchange a lane has one page.  (131,000 pages' bounds of 128 dims, 67 MB, and
// 4 heads: 28 us, issue slots 55% busy; four pages at half the occupancy took 12 us
// more.  From L2 21 us, with 8 heads 32, with 16 heads 55: instructions bound it.)
// ---------------------------------------------------------------------------
namespace pgsc {
constexpr int THREADS = 256;
constexpr int U = 2;                              // pages of a half-warp
constexpr int PPB = THREADS / 16 * U;             // pages of a block at a time
}  // namespace pgsc

// the N = D / 16 elements of lane l of 16, in pieces of 16 bytes
template <typename T, int D>
struct Sixteenth {
  static constexpr int N = D / 16;
  static constexpr int E = N * sizeof(T) < 16 ? N : 16 / sizeof(T);    // elements of a piece
  __device__ __forceinline__ static int dim(int l, int i) { return (i / E) * 16 * E + l * E + i % E; }
  __device__ __forceinline__ static void load(const T* row, int l, float (&x)[N]) {
#pragma unroll
    for (int j = 0; j < N / E; ++j) {
      const T* at = row + j * 16 * E + l * E;
      if constexpr (sizeof(T) == 4) {
        const float4 v = *reinterpret_cast<const float4*>(at);
        x[4 * j] = v.x; x[4 * j + 1] = v.y; x[4 * j + 2] = v.z; x[4 * j + 3] = v.w;
      } else {
        uint32_t w[E / 2];
        if constexpr (E == 8) {
          const uint4 v = *reinterpret_cast<const uint4*>(at);
          w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(at);
          w[0] = v.x; w[1] = v.y;
        }
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
          x[2 * i] = __uint_as_float(w[i] << 16);
          x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
      }
    }
  }
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T, int D>
__global__ void __launch_bounds__(pgsc::THREADS, 4) page_scores_kernel(ScoresArgs a, int G) {
  using namespace pgsc;
  using Row = Sixteenth<T, D>;
  constexpr int N = Row::N;
  extern __shared__ __align__(16) float sq[];    // [G][16][N]: lane l's dims together
  paged_begin();
  const int g = blockIdx.y % a.Hkv, b = blockIdx.y / a.Hkv;
  const int ps = 1 << a.ps_log2;
  const int len = min(max(a.seq_lens[b], 0), a.W << a.ps_log2);
  const int np = (len + ps - 1) >> a.ps_log2;
  const T* q = static_cast<const T*>(a.q) + b * a.q_b + (long long)g * G * a.q_h;
  for (int e = threadIdx.x; e < G * D; e += THREADS) {
    const int h = e / D, l = e % D / N, i = e % N;
    sq[e] = widen(q[(long long)h * a.q_h + Row::dim(l, i)]);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, l = lane & 15;
  const bool b0 = l & 8;
  const int mine = b0 ? 1 : 0;
  float* out = a.scores + (size_t)blockIdx.y * a.W;
  const int32_t* table = a.table + (size_t)b * a.table_stride;
  for (int p0 = blockIdx.x * PPB; p0 < a.W; p0 += gridDim.x * PPB) {
    const int first = p0 + threadIdx.x / 16 * U;
    float lo[U][N], hi[U][N];
    uint32_t live = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int page = first + u < np ? table[first + u] : -1;
      const bool ok = page >= 0 && page < a.num_pages;
      live |= (uint32_t)ok << u;
#pragma unroll
      for (int i = 0; i < N; ++i) lo[u][i] = hi[u][i] = 0.f;
      if (ok) {
        const T* x = static_cast<const T*>(a.bounds) + ((long long)page * a.Hkv + g) * 2 * D;
        Row::load(x, l, lo[u]);
        Row::load(x + D, l, hi[u]);
      }
    }
    if (__any_sync(0xffffffffu, live != 0)) {
      float best = -CUDART_INF_F;
      bool nan = false;
      for (int h = 0; h < G; ++h) {
        float qd[N], s[U];
#pragma unroll
        for (int j = 0; j < N / 4; ++j)
          *reinterpret_cast<float4*>(qd + 4 * j) = *reinterpret_cast<const float4*>(sq + h * D + l * N + 4 * j);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          s[u] = 0.f;
#pragma unroll
          for (int i = 0; i < N; ++i) s[u] = fmaf(qd[i], qd[i] < 0.f ? lo[u][i] : hi[u][i], s[u]);
        }
        // keep one page and send the other's sum
        float x = (b0 ? s[1] : s[0]) + __shfl_xor_sync(0xffffffffu, b0 ? s[0] : s[1], 8);
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        nan |= x != x;
        best = fmaxf(best, x);
      }
      if (nan) best = CUDART_NAN_F;
      if ((l & 7) == 0 && first + mine < a.W) out[first + mine] = live >> mine & 1 ? best : -CUDART_INF_F;
    } else if ((l & 7) == 0 && first + mine < a.W) {
      out[first + mine] = -CUDART_INF_F;
    }
  }
}

cudaError_t launch_page_scores(const ScoresArgs& a, bool bf16, cudaStream_t st) {
  const int G = a.Hq / a.Hkv, rows = a.B * a.Hkv;
  const int gx = max(1, min((a.W + pgsc::PPB - 1) / pgsc::PPB, num_sms() * 8 / rows));
  const dim3 grid(gx, rows);
  const size_t smem = (size_t)G * a.D * sizeof(float);
  auto go = [&](auto kern) -> cudaError_t { return paged_launch(kern, grid, pgsc::THREADS, smem, st, a, G); };
  if (bf16) return a.D == 64 ? go(page_scores_kernel<__nv_bfloat16, 64>) : go(page_scores_kernel<__nv_bfloat16, 128>);
  return a.D == 64 ? go(page_scores_kernel<float, 64>) : go(page_scores_kernel<float, 128>);
}

// ---------------------------------------------------------------------------
// selection.  A block per (sequence, kv head).  Scores become 32-bit keys of
// the same order, kept in shared memory 8192 at a time; three passes of 11,
// 11 and 10 bits narrow down the K-th largest key (the block sums a histogram of
// 2048 bins from the top), and one ordered pass writes the pages above it and the
// first ones equal to it.  Latency-bound: a list is a few KB (48 lists of up to 4096:
// 8 us, whether the keys fall into 85 bins of the first pass, into two, or are all
// alike; with four passes of 8 bits over 256 bins that one thread summed, 26 us).
// ---------------------------------------------------------------------------
namespace pgse {
constexpr int THREADS = 1024;
constexpr int NW = THREADS / 32;
constexpr int TILE = 8192;             // keys in shared memory
constexpr int BINS = 2048;
}  // namespace pgse

// Order-preserving key: pages that are always kept first, then NaN, then by value (-0 equal to 0).
__device__ __forceinline__ uint32_t select_key(const SelectArgs& a, float v, int i, int np) {
  if (i < a.keep_first || i >= np - a.keep_last) return 0xffffffffu;
  if (v != v) return 0xfffffffeu;
  const uint32_t u = __float_as_uint(v + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sum over the block (ends with every thread past its reads of s_warp).
__device__ __forceinline__ uint32_t select_scan(uint32_t x, uint32_t* s_warp, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  uint32_t w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += up;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const uint32_t before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
  __syncthreads();
  return incl - x + (warp ? before : 0u);
}

__global__ void __launch_bounds__(pgse::THREADS, 1) page_select_kernel(SelectArgs a) {
  using namespace pgse;
  __shared__ uint32_t s_key[TILE];
  __shared__ int hist[BINS];
  __shared__ uint32_t s_warp[NW];
  __shared__ uint32_t s_digit;
  __shared__ int s_need;
  paged_begin();
  const int row = blockIdx.x, tid = threadIdx.x;
  const int b = row / a.Hkv, ps = 1 << a.ps_log2;
  const int len = min(max(a.seq_lens[b], 0), a.W << a.ps_log2);
  const int np = (len + ps - 1) >> a.ps_log2;
  const float* x = a.scores + (size_t)row * a.W;
  int32_t* sel = a.sel + (size_t)row * a.K;
  const int n = min(np, a.K);
  if (tid == 0) a.n_sel[row] = n;
  for (int i = n + tid; i < a.K; i += THREADS) sel[i] = -1;
  if (np <= a.K) {
    for (int i = tid; i < np; i += THREADS) sel[i] = i;
    return;
  }
  const int ntiles = (np + TILE - 1) / TILE;
  int held = -1;       // the tile in shared memory
  auto hold = [&](int t) {
    if (held == t) return;
    __syncthreads();   // the tile before has been read
    const int i0 = t * TILE, m = min(TILE, np - i0);
#pragma unroll 4
    for (int i = tid; i < m; i += THREADS) s_key[i] = select_key(a, x[i0 + i], i0 + i, np);
    held = t;
    __syncthreads();
  };
  // the K-th largest key: its top bits so far, and how many of the keys with these top bits are wanted
  uint32_t prefix = 0;
  int need = a.K;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digit_mask = pass == 2 ? 1023u : 2047u;
    for (int i = tid; i < BINS; i += THREADS) hist[i] = 0;
    __syncthreads();
    for (int t = 0; t < ntiles; ++t) {
      hold(t);
      const int m = min(TILE, np - t * TILE);
      for (int i = tid; i < m; i += THREADS) {
        const uint32_t k = s_key[i];
        const bool in = pass == 0 || (k >> (shift + (pass == 2 ? 10 : 11))) == (prefix >> (shift + (pass == 2 ? 10 : 11)));
        if (in) atomicAdd(&hist[(k >> shift) & digit_mask], 1);
      }
    }
    __syncthreads();
    // thread t holds bins 2047 - 2t and 2046 - 2t; `above` keys lie in higher bins
    const int hi = hist[BINS - 1 - 2 * tid], lo = hist[BINS - 2 - 2 * tid];
    uint32_t total;
    const int above = (int)select_scan((uint32_t)(hi + lo), s_warp, &total);
    if (above < need && need <= above + hi + lo) {
      const bool upper = need <= above + hi;
      s_digit = (uint32_t)(upper ? BINS - 1 - 2 * tid : BINS - 2 - 2 * tid);
      s_need = need - above - (upper ? 0 : hi);
    }
    __syncthreads();
    prefix |= s_digit << shift;
    need = s_need;
  }
  // keys above `prefix`, and the first `need` equal to it, in index order: a thread takes 8 in a row
  int above = 0, equal = 0;      // before this tile
  for (int t = 0; t < ntiles; ++t) {
    hold(t);
    constexpr int PER = TILE / THREADS;
    const int m = min(TILE, np - t * TILE);
    uint32_t mine = 0;           // keys equal to prefix : keys above it
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = tid * PER + i;
      const uint32_t k = at < m ? s_key[at] : 0u;
      mine += (at < m && k > prefix ? 1u : 0u) + (at < m && k == prefix ? 0x10000u : 0u);
    }
    uint32_t total;
    const uint32_t before = select_scan(mine, s_warp, &total);
    int rg = above + (int)(before & 0xffffu), re = equal + (int)(before >> 16);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = tid * PER + i;
      if (at >= m) break;
      const uint32_t k = s_key[at];
      if (k > prefix) {
        sel[rg + min(re, need)] = t * TILE + at;
        ++rg;
      } else if (k == prefix) {
        if (re < need) sel[rg + re] = t * TILE + at;
        ++re;
      }
    }
    above += (int)(total & 0xffffu);
    equal += (int)(total >> 16);
  }
}

cudaError_t launch_page_select(const SelectArgs& a, cudaStream_t st) {
  return paged_launch(page_select_kernel, a.B * a.Hkv, pgse::THREADS, 0, st, a);
}

}  // namespace ra
