// How the paged decode kernels share the work, and how their pieces are joined.
//
// The keys of every (sequence, kv head, head group) -- a segment -- are cut
// into tiles of 128, and all tiles of the call, segment after segment, are
// dealt to n CTAs in n equal contiguous runs (CTA c gets tiles
// [cT/n, (c+1)T/n) of T).  Ragged batches balance whatever their lengths, one
// long sequence spreads over the whole GPU, and the lengths are read on the
// device, so a captured launch follows them.  A run covers whole segments,
// whose result is written at once, and at most two parts of segments (at its
// start and at its end), whose normalised output and lse go to the workspace;
// of the CTAs that share a segment the last to finish joins the parts in CTA
// order (the result does not depend on which CTA that is):
//   lse = m* + ln sum_p e^(lse_p - m*),  out = sum_p e^(lse_p - lse) O_p.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "paged.h"
#include "ptx.cuh"

namespace ra {

struct PagedRows {     // rows of equal-length segments: sequences, or (sequence, kv head) with a page list
  int R, mult;         // rows, segments per row
};
__device__ __forceinline__ PagedRows paged_rows(const PagedDecodeArgs& a) {
  if (a.sel) return {a.B * a.Hkv, a.ngrp};
  return {a.B, a.Hkv * a.ngrp};
}
// Valid length of a sequence (clamped, never trusted).
__device__ __forceinline__ int paged_len(const PagedDecodeArgs& a, int b) {
  return min(max(a.seq_lens[b], 0), a.W << a.ps_log2);
}
// Keys listed for row r (with a page list: whole pages; those past the length are masked later).
__device__ __forceinline__ int paged_keys(const PagedDecodeArgs& a, int r) {
  if (a.sel) return min(max(a.n_sel[r], 0), a.K) << a.ps_log2;
  return paged_len(a, r);
}
__device__ __forceinline__ int paged_tiles(const PagedDecodeArgs& a, int r) {
  return (paged_keys(a, r) + kPagedTile - 1) / kPagedTile;
}

struct PagedRun {
  int T;          // tiles of the call
  int n;          // CTAs that have work
  int t0, t1;     // this CTA's tiles
  int row;        // row that holds t0
  int row_t;      // first tile of that row
};
__device__ __forceinline__ int run_start(int T, int n, int c) { return (int)((long long)c * T / n); }
__device__ __forceinline__ int run_owner(int T, int n, int t) { return (int)(((long long)(t + 1) * n - 1) / T); }

struct PagedRunSmem {
  int warp_sum[32];
  int row, row_t, total;
};

// All threads of the CTA (a multiple of 32, at most 1024).  min_tiles: the
// fewest tiles worth a CTA of their own.
template <int kThreads>
__device__ __forceinline__ PagedRun paged_run(const PagedDecodeArgs& a, PagedRunSmem& s, int min_tiles) {
  constexpr int NW = kThreads / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedRows rows = paged_rows(a);
  // total number of tiles; the first kThreads rows stay in registers
  const int mine = tid < rows.R ? paged_tiles(a, tid) : 0;
  int sum = mine;
  for (int r = tid + kThreads; r < rows.R; r += kThreads) sum += paged_tiles(a, r);
  sum = __reduce_add_sync(0xffffffffu, sum);
  if (lane == 0) s.warp_sum[warp] = sum;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) total += s.warp_sum[w];
  PagedRun run;
  run.T = total * rows.mult;
  run.n = min((int)gridDim.x, max(1, run.T / min_tiles));
  run.row = run.row_t = 0;
  const int c = blockIdx.x;
  if (run.T == 0 || c >= run.n) {
    run.t0 = run.t1 = 0;
    return run;
  }
  run.t0 = run_start(run.T, run.n, c);
  run.t1 = run_start(run.T, run.n, c + 1);
  // the row that holds t0
  const int want = run.t0 / rows.mult;    // tile index counted once per row
  int base = 0;
  for (int r0 = 0; r0 < rows.R; r0 += kThreads) {
    const int r = r0 + tid;
    const int nt = r0 == 0 ? mine : (r < rows.R ? paged_tiles(a, r) : 0);
    int incl = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    __syncthreads();    // warp_sum is free
    if (lane == 31) s.warp_sum[warp] = incl;
    __syncthreads();
    int before = base, chunk = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < warp) before += s.warp_sum[w];
      chunk += s.warp_sum[w];
    }
    const int hi = before + incl, lo = hi - nt;
    if (lo <= want && want < hi) {
      s.row = r;
      s.row_t = lo * rows.mult;
    }
    base += chunk;
    if (want < base) break;    // the same in every thread
  }
  __syncthreads();
  run.row = s.row;
  run.row_t = s.row_t;
  return run;
}

// Walks a run's pieces: [a, b) tiles of one segment.
struct PagedPiece {
  int row, sub;    // row and segment of the row
  int nt;          // tiles of the whole segment
  int a, b;        // this piece's tiles
  int seg_t;       // first tile of the segment, counted over the call
};
struct PagedWalk {
  int t, t1, row, row_t;
  __device__ __forceinline__ explicit PagedWalk(const PagedRun& r) : t(r.t0), t1(r.t1), row(r.row), row_t(r.row_t) {}
  __device__ __forceinline__ bool next(const PagedDecodeArgs& a, const PagedRows& rows, PagedPiece& p) {
    if (t >= t1) return false;
    int nt = paged_tiles(a, row);
    while (t - row_t >= nt * rows.mult) {    // never past the last row: t < t1 <= T
      row_t += nt * rows.mult;
      ++row;
      nt = paged_tiles(a, row);
    }
    const int o = t - row_t;
    p.row = row;
    p.sub = o / nt;
    p.nt = nt;
    p.a = o - p.sub * nt;
    p.b = min(nt, p.a + (t1 - t));
    p.seg_t = row_t + p.sub * nt;
    t += p.b - p.a;
    return true;
  }
};
// Sequence, kv head and first query head (of the call's Hq) of a piece.
struct PagedHead {
  int b, g, h0, nh;
};
__device__ __forceinline__ PagedHead paged_head(const PagedDecodeArgs& a, int row, int sub, int group_heads) {
  PagedHead p;
  int grp;
  if (a.sel) {
    p.b = row / a.Hkv;
    p.g = row - p.b * a.Hkv;
    grp = sub;
  } else {
    p.b = row;
    p.g = sub / a.ngrp;
    grp = sub - p.g * a.ngrp;
  }
  p.h0 = p.g * a.G + grp * group_heads;
  p.nh = min(group_heads, a.G - grp * group_heads);
  return p;
}

// Pool page and number of valid keys of the keys [k0, k0 + n) of a segment
// (n divides the page size or the reverse; the keys lie in one page).  Keys
// past the length, listed pages outside the sequence and table entries
// outside the pool have no valid key.
struct PagedSpan {
  int page, in_page, valid;
};
__device__ __forceinline__ PagedSpan paged_span(const PagedDecodeArgs& a, int b, int g, int len, int k0, int n) {
  PagedSpan s;
  int lp = k0 >> a.ps_log2;
  s.in_page = k0 & ((1 << a.ps_log2) - 1);
  s.page = -1;
  s.valid = 0;
  if (a.sel) {
    const int r = b * a.Hkv + g;
    if (lp >= min(max(a.n_sel[r], 0), a.K)) return s;
    lp = a.sel[(size_t)r * a.K + lp];
    if (lp < 0 || lp >= a.W) return s;
  }
  s.valid = min(max(len - (lp << a.ps_log2) - s.in_page, 0), n);
  if (s.valid > 0) {
    s.page = a.table[(size_t)b * a.table_stride + lp];
    if (s.page < 0 || s.page >= a.num_pages) s.valid = 0;
  }
  return s;
}

__device__ __forceinline__ void paged_store(const PagedDecodeArgs& a, size_t at, float x) {
  if (a.out_fp32)
    static_cast<float*>(a.out)[at] = x;
  else
    static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(x);
}

// out = 0, lse = -inf for the rows without a key (threads tid of nthreads of every CTA).
__device__ __forceinline__ void paged_empty_rows(const PagedDecodeArgs& a, int tid, int nthreads) {
  const PagedRows rows = paged_rows(a);
  for (int r = blockIdx.x; r < rows.R; r += gridDim.x) {
    if (paged_keys(a, r) > 0) continue;
    // a row's query heads: all of the sequence, or the kv head's
    const size_t h0 = a.sel ? (size_t)r * a.G : (size_t)r * a.Hq;
    const int nh = a.sel ? a.G : a.Hq;
    for (int e = tid; e < nh * a.D; e += nthreads) paged_store(a, h0 * a.D + e, 0.f);
    if (a.out_lse)
      for (int e = tid; e < nh; e += nthreads) a.out_lse[h0 + e] = -CUDART_INF_F;
  }
}

// Workspace slot of CTA c's part of the segment that starts at tile seg_t:
// slot 0 if the CTA's run starts inside the segment (or with it), else 1.
__device__ __forceinline__ float* paged_part(const PagedDecodeArgs& a, const PagedRun& run, int c, int seg_t) {
  const int slot = run_start(run.T, run.n, c) >= seg_t ? 0 : 1;
  return a.ws_part + (size_t)(c * 2 + slot) * kPagedHeads * (a.D + 1);
}

// Joins the parts of a segment (its CTAs c0..c1) and writes the result.
// Called by kThreads threads after the acquire of the last arrival.
template <int kThreads>
__device__ __forceinline__ void paged_join(const PagedDecodeArgs& a, const PagedRun& run, const PagedPiece& pc,
                                           const PagedHead& hd, int c0, int c1, int tid) {
  for (int e = tid; e < hd.nh * a.D; e += kThreads) {
    const int h = e / a.D, d = e - h * a.D;
    float mx = -CUDART_INF_F;
    for (int c = c0; c <= c1; ++c)
      mx = fmaxf(mx, __ldcg(paged_part(a, run, c, pc.seg_t) + kPagedHeads * a.D + h));
    float L = 0.f, acc = 0.f;
    for (int c = c0; c <= c1; ++c) {
      const float* part = paged_part(a, run, c, pc.seg_t);
      const float lse = __ldcg(part + kPagedHeads * a.D + h);
      const float w = lse == -CUDART_INF_F ? 0.f : expf(lse - mx);   // a part without a key adds nothing
      L += w;
      acc = fmaf(w, __ldcg(part + h * a.D + d), acc);
    }
    const size_t bh = (size_t)hd.b * a.Hq + hd.h0 + h;
    paged_store(a, bh * a.D + d, L == 0.f ? 0.f : acc / L);
    if (d == 0 && a.out_lse) a.out_lse[bh] = L == 0.f ? -CUDART_INF_F : mx + logf(L);
  }
}

}  // namespace ra
