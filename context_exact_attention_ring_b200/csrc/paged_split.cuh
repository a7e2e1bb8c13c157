// How the paged decode kernels share the work, and how their pieces are joined.
//
// The keys of every (sequence, kv head, head group) -- a segment -- are cut
// into tiles of 128, and all tiles of the call, segment after segment, are
// dealt to n CTAs in n contiguous runs of as many units (a unit is a tile or a
// segment's fixed cost), give or take one.  Ragged batches balance whatever their lengths, one
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

#include "paged.cuh"

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

// Segments of up to this many tiles are not split: the CTA that has their
// first unit takes them whole.  Joining costs some 5 us at the end of a call
// (partial results to L2, an atomic, the parts back), four tiles 3 us.
constexpr int kPagedWhole = 4;

// Units of work of a row's segments: its tiles, and what starting and
// finishing a segment costs, in tiles (a run's boundary in that tail belongs
// to no tile).
__device__ __forceinline__ int paged_units(int tiles, int seg_cost) { return tiles ? tiles + seg_cost : 0; }

struct PagedRun {
  int T;          // units of the call
  int n;          // CTAs that have work
  int q, r;       // T = n q + r: the first r CTAs get q + 1 units, the others q
  int t0, t1;     // this CTA's units
  int row;        // row that holds t0
  int row_t;      // first unit of that row
};
__device__ __forceinline__ int run_start(const PagedRun& r, int c) { return c * r.q + min(c, r.r); }
__device__ __forceinline__ int run_owner(const PagedRun& r, int t) {
  const int big = r.r * (r.q + 1);
  return t < big ? t / (r.q + 1) : r.r + (t - big) / r.q;
}

struct PagedRunSmem {
  int units[32], rows[32], more[32];    // per warp
  int row, row_t;
};

// The number of CTAs for run.T units in segs segments, and this CTA's run.
// parts_per_tile: how many parts a segment may be cut into for every tile of
// a part.  Joining takes as long as a tile for every parts_per_tile parts, so
// that the time with n parts, T / n + n / parts_per_tile, is shortest at
// n^2 = parts_per_tile T.
__device__ __forceinline__ void paged_cut(PagedRun& run, int segs, int seg_cost, int parts_per_tile) {
  const int tiles = run.T - segs * seg_cost, c = blockIdx.x;
  run.n = max(1, min(min((int)gridDim.x, tiles), (int)sqrtf((float)parts_per_tile * tiles * segs)));
  run.row = run.row_t = run.q = run.r = run.t0 = run.t1 = 0;
  if (run.T == 0 || c >= run.n) return;
  run.q = run.T / run.n;
  run.r = run.T - run.n * run.q;
  run.t0 = run_start(run, c);
  run.t1 = run_start(run, c + 1);
}

// The plan by all threads of the CTA (a multiple of 32, at most 1024).
// mine: the tiles of row threadIdx.x (paged_first_tiles), loaded earlier.
__device__ __forceinline__ int paged_first_tiles(const PagedDecodeArgs& a) {
  return (int)threadIdx.x < paged_rows(a).R ? paged_tiles(a, threadIdx.x) : 0;
}
template <int kThreads>
__device__ __forceinline__ PagedRun paged_run(const PagedDecodeArgs& a, PagedRunSmem& s, int mine, int seg_cost,
                                              int parts_per_tile) {
  constexpr int NW = kThreads / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedRows rows = paged_rows(a);
  auto scan = [&](int x) {    // inclusive, over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += up;
    }
    return x;
  };
  // the first kThreads rows' units up to each row, and the sums over all rows
  const int units0 = paged_units(mine, seg_cost), incl0 = scan(units0);
  int some = __popc(__ballot_sync(0xffffffffu, mine > 0)), more_tiles = 0, more_rows = 0;
  for (int r = tid + kThreads; r < rows.R; r += kThreads) {
    const int nt = paged_tiles(a, r);
    more_tiles += nt;
    more_rows += nt > 0;
  }
  if (rows.R > kThreads) {
    more_tiles = __reduce_add_sync(0xffffffffu, more_tiles);
    more_rows = __reduce_add_sync(0xffffffffu, more_rows);
  }
  if (lane == 31) {
    s.units[warp] = incl0;
    s.rows[warp] = some + more_rows;
    s.more[warp] = more_tiles + more_rows * seg_cost;
  }
  __syncthreads();
  int units = 0, segs = 0, more = 0, before = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w == warp) before = units;
    units += s.units[w];
    segs += s.rows[w];
    more += s.more[w];
  }
  PagedRun run;
  run.T = (units + more) * rows.mult;
  paged_cut(run, segs * rows.mult, seg_cost, parts_per_tile);
  if (run.t0 == run.t1) return run;
  // the row that holds t0
  const int want = run.t0 / rows.mult;    // units counted once per row
  int hi = before + incl0, lo = hi - units0, base = units;
  if (lo <= want && want < hi) {
    s.row = tid;
    s.row_t = lo * rows.mult;
  }
  for (int r0 = kThreads; r0 < rows.R && want >= base; r0 += kThreads) {    // the same in every thread
    const int r = r0 + tid;
    const int nu = paged_units(r < rows.R ? paged_tiles(a, r) : 0, seg_cost), incl = scan(nu);
    __syncthreads();    // s.units is free
    if (lane == 31) s.units[warp] = incl;
    __syncthreads();
    hi = base + incl;
    int chunk = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < warp) hi += s.units[w];
      chunk += s.units[w];
    }
    lo = hi - nu;
    if (lo <= want && want < hi) {
      s.row = r;
      s.row_t = lo * rows.mult;
    }
    base += chunk;
  }
  __syncthreads();
  run.row = s.row;
  run.row_t = s.row_t;
  return run;
}

// The same for at most 32 rows, by every warp on its own (no barrier): mine is
// the tiles of row `lane`.
__device__ __forceinline__ PagedRun paged_run_warp(const PagedDecodeArgs& a, int mine, int seg_cost,
                                                   int parts_per_tile) {
  const int lane = threadIdx.x & 31;
  const PagedRows rows = paged_rows(a);
  const int nu = paged_units(mine, seg_cost);
  int hi = nu;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, hi, o);
    if (lane >= o) hi += up;
  }
  PagedRun run;
  const int segs = __popc(__ballot_sync(0xffffffffu, mine > 0)) * rows.mult;
  run.T = __shfl_sync(0xffffffffu, hi, 31) * rows.mult;
  paged_cut(run, segs, seg_cost, parts_per_tile);
  if (run.t0 < run.t1) {
    const int want = run.t0 / rows.mult;
    run.row = __ffs(__ballot_sync(0xffffffffu, want < hi)) - 1;      // the first whose units end past it
    run.row_t = __shfl_sync(0xffffffffu, hi - nu, run.row) * rows.mult;
  }
  return run;
}

// Walks a run's pieces: [a, b) tiles of one segment.
struct PagedPiece {
  int row, sub;    // row and segment of the row
  int nt;          // tiles of the whole segment
  int a, b;        // this piece's tiles
  int seg_t;       // first unit of the segment, counted over the call
};
struct PagedWalk {
  int t1, seg_cost;
  int row, sub, nt, nu, seg_t, from;    // the next segment: its tiles, units, first unit; the unit of it to begin at
  __device__ __forceinline__ PagedWalk(const PagedDecodeArgs& a, const PagedRows& rows, const PagedRun& r, int cost)
      : t1(r.t1), seg_cost(cost), row(r.row), sub(0), nt(0), nu(0), seg_t(r.row_t), from(0) {
    if (r.t0 >= t1) {
      seg_t = t1;
      return;
    }
    nt = paged_tiles(a, row);
    nu = paged_units(nt, seg_cost);
    from = r.t0 - seg_t;
    sub = from / nu;
    seg_t += sub * nu;
    from -= sub * nu;
  }
  __device__ __forceinline__ bool next(const PagedDecodeArgs& a, const PagedRows& rows, PagedPiece& p) {
    while (seg_t < t1) {
      const bool whole = nt <= kPagedWhole;
      p.row = row;
      p.sub = sub;
      p.nt = nt;
      p.seg_t = seg_t;
      p.a = from;
      p.b = whole ? (from > 0 ? 0 : nt) : min(nt, t1 - seg_t);
      from = 0;
      seg_t += nu;
      if (seg_t < t1 && ++sub == rows.mult) {      // a row with keys follows: t1 <= T
        sub = 0;
        do nt = paged_tiles(a, ++row);
        while (nt == 0);
        nu = paged_units(nt, seg_cost);
      }
      if (p.a < p.b) return true;    // else the tail of a segment, or the rest of one that is not split
    }
    return false;
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
    p.g = a.ngrp == 1 ? sub : sub / a.ngrp;
    grp = sub - p.g * a.ngrp;
  }
  p.h0 = p.g * a.G + grp * group_heads;
  p.nh = min(group_heads, a.G - grp * group_heads);
  return p;
}

// Pool page and number of valid keys of the keys [k0, k0 + n) of a segment
// (n divides the page size or the reverse; the keys lie in one page).  Keys
// past the length, listed pages outside the sequence and table entries
// outside the pool have no valid key; the last is left to paged_valid, so that
// the table entry may be on its way meanwhile.
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
  if (s.valid > 0) s.page = a.table[(size_t)b * a.table_stride + lp];
  return s;
}
__device__ __forceinline__ int paged_valid(const PagedDecodeArgs& a, const PagedSpan& s) {
  return (unsigned)s.page < (unsigned)a.num_pages ? s.valid : 0;
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

// Workspace slot of this CTA's part of the segment that starts at tile seg_t:
// 0 if its run starts inside the segment (or with it), else 1.  Only the
// first CTA of a segment can have started before it.
__device__ __forceinline__ float* paged_part(const PagedDecodeArgs& a, int c, int slot) {
  return a.ws_part + (size_t)(c * 2 + slot) * kPagedHeads * (a.D + 1);
}

// Joins the parts of a segment (of its CTAs c0..c1) and writes the result, 4
// heads at a time.  Called by kThreads threads after the acquire of the last
// arrival; sync() is their barrier.  A row of D dims takes D / 4 lanes; the
// groups of lanes share out the parts, and a lane has 4 parts of 4 heads in
// flight before it needs the first weight.  The weights come from the lse
// values meanwhile: a warp to a head, a lane to every 32nd part.  The groups'
// sums meet in shared memory.  (Of 9 to 16 heads, 8 at a time, the groups share
// out the heads instead, which needs no shared memory for the sums.)  (One thread per output looking the parts up one
// after the other took 60 us of a 65 us call.)
template <int kThreads, int G, int D>
struct PagedJoin {
  static constexpr int NG = kThreads / (D / 4);                 // groups of lanes
  static constexpr bool BY_HEAD = G > 8;                        // groups over heads, not parts
  static constexpr int H = BY_HEAD ? 8 : G < 4 ? G : 4;         // heads at a time
  static constexpr int HL = BY_HEAD ? (H + NG - 1) / NG : H;    // heads of a lane
  static constexpr int U = BY_HEAD ? 8 : kThreads > 256 ? 1 : 4;    // parts a lane has in flight
  struct Smem {
    float w[kPagedMaxCtas * H];
    alignas(16) float4 o[BY_HEAD ? 1 : NG][BY_HEAD ? 1 : H][BY_HEAD ? 1 : D / 4];
  };
};
template <int kThreads, int G, int D, typename Sync>
__device__ __forceinline__ void paged_join(const PagedDecodeArgs& a, const PagedRun& run, const PagedPiece& pc,
                                           const PagedHead& hd, int c0, int c1, int tid,
                                           typename PagedJoin<kThreads, G, D>::Smem& js, Sync sync) {
  using J = PagedJoin<kThreads, G, D>;
  constexpr int NW = kThreads / 32, H = J::H, HL = J::HL, U = J::U;
  constexpr int CS = J::BY_HEAD ? 1 : J::NG;                    // a lane's parts: cf, cf + CS, ...
  constexpr int KV = (kPagedMaxCtas + 31) / 32;                 // lse values per lane
  const int warp = tid >> 5, lane = tid & 31;
  const int n = c1 - c0 + 1;
  const int slot0 = run_start(run, c0) >= pc.seg_t ? 0 : 1;
  const int step = 2 * kPagedHeads * (D + 1);
  const float* first = paged_part(a, c0, slot0);
  const float* rest = paged_part(a, c0, 0);                     // part i > 0 at rest + i step
  const size_t bh0 = (size_t)hd.b * a.Hq + hd.h0;
  const int d4 = tid % (D / 4), grp = tid / (D / 4);
  const int cf = J::BY_HEAD ? 0 : grp, hl = J::BY_HEAD ? grp * HL : 0;
  for (int hb = 0; hb < hd.nh; hb += H) {
    const int mine = min(HL, min(H, hd.nh - hb) - hl);          // this lane's heads, from hb + hl on
    float4 x[U][HL], acc[HL];
    auto fetch = [&](int c) {
#pragma unroll
      for (int u = 0; u < U; ++u, c += CS) {
        const float4* part = reinterpret_cast<const float4*>(c ? rest + c * step : first) + (hb + hl) * (D / 4) + d4;
#pragma unroll
        for (int h = 0; h < HL; ++h)
          x[u][h] = c < n && h < mine ? __ldcg(part + h * (D / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    fetch(cf);
    for (int h = warp; h < H && hb + h < hd.nh; h += NW) {
      float w[KV], mx = -CUDART_INF_F;
#pragma unroll
      for (int k = 0; k < KV; ++k) {
        const int c = lane + 32 * k;
        w[k] = c < n ? __ldcg((c ? rest + c * step : first) + kPagedHeads * D + hb + h) : -CUDART_INF_F;
      }
#pragma unroll
      for (int k = 0; k < KV; ++k) mx = fmaxf(mx, w[k]);
#pragma unroll
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      float L = 0.f;
#pragma unroll
      for (int k = 0; k < KV; ++k) {
        w[k] = w[k] == -CUDART_INF_F ? 0.f : expf(w[k] - mx);   // a part without a key adds nothing
        L += w[k];
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
      const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
      for (int k = 0; k < KV; ++k)
        if (lane + 32 * k < n) js.w[(lane + 32 * k) * H + h] = w[k] * inv;
      if (lane == 0 && a.out_lse) a.out_lse[bh0 + hb + h] = L == 0.f ? -CUDART_INF_F : mx + logf(L);
    }
#pragma unroll
    for (int h = 0; h < HL; ++h) acc[h] = make_float4(0.f, 0.f, 0.f, 0.f);
    sync();
    for (int c = cf; c < n; c += U * CS) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c + u * CS < n)
#pragma unroll
          for (int h = 0; h < HL; ++h) {
            const float wv = h < mine ? js.w[(c + u * CS) * H + hl + h] : 0.f;
            acc[h].x = fmaf(wv, x[u][h].x, acc[h].x);
            acc[h].y = fmaf(wv, x[u][h].y, acc[h].y);
            acc[h].z = fmaf(wv, x[u][h].z, acc[h].z);
            acc[h].w = fmaf(wv, x[u][h].w, acc[h].w);
          }
      if (c + U * CS < n) fetch(c + U * CS);
    }
    if constexpr (J::BY_HEAD) {
#pragma unroll
      for (int h = 0; h < HL; ++h)
        if (h < mine) {
          const size_t to = (bh0 + hb + hl + h) * D + 4 * d4;
          paged_store(a, to, acc[h].x);
          paged_store(a, to + 1, acc[h].y);
          paged_store(a, to + 2, acc[h].z);
          paged_store(a, to + 3, acc[h].w);
        }
    } else {
#pragma unroll
      for (int h = 0; h < H; ++h) js.o[grp][h][d4] = acc[h];
      sync();
      const int ne = min(H, hd.nh - hb) * D;
      for (int e = tid; e < ne; e += kThreads) {
        float o = 0.f;
#pragma unroll
        for (int p = 0; p < J::NG; ++p) o += reinterpret_cast<const float*>(js.o[p])[e];
        paged_store(a, (bh0 + hb) * D + e, o);
      }
    }
    sync();     // js is free
  }
}

}  // namespace ra
