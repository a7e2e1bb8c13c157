// Which pages of a long cache a query needs: bounds, scores, selection.
//
// bounds   per page and kv head the elementwise minimum lo and maximum hi of
//          the page's valid keys (comparisons only: exact in the cache's type).
// scores   score(page) = max over the heads h of the group of
//            sum_d max(q_hd lo_d, q_hd hi_d) >= max_h max_{key in page} q_h . k,
//          so no key of a page scores above it.
// select   the K best pages of a (sequence, kv head), in ascending order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "kernels.h"
#include "paged.cuh"

namespace ra {

// ---------------------------------------------------------------------------
// bounds.  A copy-like pass over the keys: a block takes one page at a time of
// one sequence, a thread a 4-element column of the page's rows of all heads.
// ---------------------------------------------------------------------------
namespace pgb {
constexpr int THREADS = 256;
}

// minimum and maximum that keep a NaN
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ void load4(const float* p, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&x)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  x[0] = __uint_as_float(v.x << 16);
  x[1] = __uint_as_float(v.x & 0xffff0000u);
  x[2] = __uint_as_float(v.y << 16);
  x[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
// exact: the values came from bf16
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&x)[4]) {
  *reinterpret_cast<uint2*>(p) =
      make_uint2((__float_as_uint(x[0]) >> 16) | (__float_as_uint(x[1]) & 0xffff0000u),
                 (__float_as_uint(x[2]) >> 16) | (__float_as_uint(x[3]) & 0xffff0000u));
}

template <typename T>
__global__ void __launch_bounds__(pgb::THREADS) page_bounds_kernel(BoundsArgs a) {
  paged_begin();
  const int b = blockIdx.y, ps = 1 << a.ps_log2;
  const int len = min(max(a.seq_lens[b], 0), a.W << a.ps_log2);
  const int start = a.start_lens ? max(a.start_lens[b], 0) : 0;
  const int np = (len + ps - 1) >> a.ps_log2;
  const int nc = a.Hkv * a.D / 4;
  for (int p = (start >> a.ps_log2) + blockIdx.x; p < np; p += gridDim.x) {
    const int page = a.table[(size_t)b * a.table_stride + p];
    if (page < 0 || page >= a.num_pages) continue;
    const int rows = min(ps, len - (p << a.ps_log2));
    for (int c = threadIdx.x; c < nc; c += pgb::THREADS) {
      const int h = c * 4 / a.D, d = c * 4 - h * a.D;
      const T* k = static_cast<const T*>(a.k) + (long long)page * a.pool.page + (long long)h * a.pool.head + d;
      float lo[4], hi[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] = CUDART_INF_F;
        hi[i] = -CUDART_INF_F;
      }
#pragma unroll 8
      for (int r = 0; r < rows; ++r) {
        float x[4];
        load4(k + (long long)r * a.pool.token, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = min_nan(lo[i], x[i]);
          hi[i] = max_nan(hi[i], x[i]);
        }
      }
      T* o = static_cast<T*>(a.bounds) + ((long long)page * a.Hkv + h) * 2 * a.D + d;
      store4(o, lo);
      store4(o + a.D, hi);
    }
  }
}

cudaError_t launch_page_bounds(const BoundsArgs& a, cudaStream_t st) {
  // enough blocks to fill the GPU; each walks its share of a sequence's pages
  const int gx = max(1, min(a.W, num_sms() * 16 / a.B));
  const dim3 grid(gx, a.B);
  if (a.elem_bytes == 2) return paged_launch(page_bounds_kernel<__nv_bfloat16>, grid, pgb::THREADS, 0, st, a);
  return paged_launch(page_bounds_kernel<float>, grid, pgb::THREADS, 0, st, a);
}

// ---------------------------------------------------------------------------
// scores.  Bound by the bytes of the bounds: a warp takes a page, a lane D/32
// of its dims; the group's queries wait in shared memory.
// ---------------------------------------------------------------------------
namespace pgsc {
constexpr int THREADS = 256;
}

template <typename T>
__device__ __forceinline__ float widen(T x);
template <>
__device__ __forceinline__ float widen(float x) { return x; }
template <>
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T, int D>
__global__ void __launch_bounds__(pgsc::THREADS) page_scores_kernel(ScoresArgs a, int G) {
  extern __shared__ float sq[];    // [G][D]
  paged_begin();
  const int g = blockIdx.y % a.Hkv, b = blockIdx.y / a.Hkv;
  const int ps = 1 << a.ps_log2;
  const int len = min(max(a.seq_lens[b], 0), a.W << a.ps_log2);
  const int np = (len + ps - 1) >> a.ps_log2;
  const T* q = static_cast<const T*>(a.q) + b * a.q_b + (long long)g * G * a.q_h;
  for (int e = threadIdx.x; e < G * D; e += pgsc::THREADS) sq[e] = widen(q[(long long)(e / D) * a.q_h + e % D]);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int N = D / 32, NW = pgsc::THREADS / 32;
  float* out = a.scores + (size_t)blockIdx.y * a.W;
  for (int p = blockIdx.x * NW + warp; p < a.W; p += gridDim.x * NW) {
    float best = -CUDART_INF_F;
    const int page = p < np ? a.table[(size_t)b * a.table_stride + p] : -1;
    if (page >= 0 && page < a.num_pages) {
      const T* x = static_cast<const T*>(a.bounds) + ((long long)page * a.Hkv + g) * 2 * D + lane * N;
      float lo[N], hi[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        lo[i] = widen(x[i]);
        hi[i] = widen(x[D + i]);
      }
      for (int h = 0; h < G; ++h) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float qd = sq[h * D + lane * N + i];
          s += fmaxf(qd * lo[i], qd * hi[i]);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        best = h ? max(best, s) : s;
      }
    }
    if (lane == 0) out[p] = best;
  }
}

cudaError_t launch_page_scores(const ScoresArgs& a, bool bf16, cudaStream_t st) {
  const int G = a.Hq / a.Hkv, rows = a.B * a.Hkv;
  const int gx = max(1, min((a.W + 7) / 8, num_sms() * 8 / rows));
  const dim3 grid(gx, rows);
  const size_t smem = (size_t)G * a.D * sizeof(float);
  auto go = [&](auto kern) -> cudaError_t { return paged_launch(kern, grid, pgsc::THREADS, smem, st, a, G); };
  if (bf16) return a.D == 64 ? go(page_scores_kernel<__nv_bfloat16, 64>) : go(page_scores_kernel<__nv_bfloat16, 128>);
  return a.D == 64 ? go(page_scores_kernel<float, 64>) : go(page_scores_kernel<float, 128>);
}

// ---------------------------------------------------------------------------
// selection.  A block per (sequence, kv head).  Scores become 32-bit keys of
// the same order; four passes of 8 bits each narrow down the K-th largest key,
// and one ordered pass writes the pages above it and the first ones equal to
// it.
// ---------------------------------------------------------------------------
namespace pgse {
constexpr int THREADS = 1024;
constexpr int NW = THREADS / 32;
}  // namespace pgse

// Order-preserving key: pages that are always kept first, then NaN, then by value (-0 equal to 0).
__device__ __forceinline__ uint32_t select_key(const SelectArgs& a, const float* x, int i, int np) {
  if (i < a.keep_first || i >= np - a.keep_last) return 0xffffffffu;
  const float v = x[i];
  if (v != v) return 0xfffffffeu;
  const uint32_t u = __float_as_uint(v + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(pgse::THREADS) page_select_kernel(SelectArgs a) {
  using namespace pgse;
  __shared__ int hist[256];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  __shared__ uint32_t s_warp[NW];
  paged_begin();
  const int row = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
  // the K-th largest key: its top bits so far, and how many of the keys with these top bits are wanted
  uint32_t prefix = 0;
  int need = a.K;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < np; i += THREADS) {
      const uint32_t k = select_key(a, x, i, np);
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int left = need, d = 255;
      while (d > 0 && hist[d] < left) left -= hist[d--];
      s_prefix = prefix | ((uint32_t)d << shift);
      s_need = left;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  // keys above `prefix`, and the first `need` equal to it, in index order
  int above = 0, equal = 0;      // before this chunk
  for (int i0 = 0; i0 < np; i0 += THREADS) {
    const int i = i0 + tid;
    const uint32_t k = i < np ? select_key(a, x, i, np) : 0u;
    const bool gt = i < np && k > prefix, eq = i < np && k == prefix;
    const uint32_t mine = (gt ? 1u : 0u) | (eq ? 0x10000u : 0u);
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    uint32_t before = 0, chunk = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < warp) before += s_warp[w];
      chunk += s_warp[w];
    }
    const uint32_t excl = before + incl - mine;
    const int rg = above + (int)(excl & 0xffffu), re = equal + (int)(excl >> 16);
    if (gt || (eq && re < need)) sel[rg + min(re, need)] = i;
    above += (int)(chunk & 0xffffu);
    equal += (int)(chunk >> 16);
    __syncthreads();
  }
}

cudaError_t launch_page_select(const SelectArgs& a, cudaStream_t st) {
  return paged_launch(page_select_kernel, a.B * a.Hkv, pgse::THREADS, 0, st, a);
}

}  // namespace ra
