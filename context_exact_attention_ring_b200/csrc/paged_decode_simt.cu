// Paged decode on CUDA cores: one new token per sequence against the keys in
// its cache pages,
//   out_h = sum_j softmax_j(scale q_h . k_j) v_j,   lse_h = ln sum_j e^(scale q_h . k_j),
// in one pass over the keys with a running maximum and sum.
//
// float32 caches run here (the tensor cores have no float32 product); every
// product and sum is float32.  A CTA of 8 warps takes the tiles of its run
// (paged_split.cuh) 128 keys at a time, 16 keys a warp: 16 lanes share a key
// row, so that a row is one contiguous load of the half-warp, and each lane
// keeps D/16 dims of the queries and outputs of up to 8 heads in registers.
#include <cuda_runtime.h>

#include "kernels.h"
#include "paged.h"
#include "paged_split.cuh"

namespace ra {

namespace pds {
constexpr int THREADS = 256;
constexpr int NW = THREADS / 32;
constexpr int KPW = 8;      // keys a half-warp holds at once (a tile is 8 warps x 2 x 8 keys)
constexpr int HEADS = 8;    // query heads of a group, at most
constexpr int SEG_COST = 1;         // what a segment costs besides its tiles, in tiles
constexpr int PARTS_PER_TILE = 10;  // parts joined in the time of a tile
}  // namespace pds
static_assert(pds::NW * 2 * pds::KPW == kPagedTile, "a CTA takes a tile at a time");

// Dims of a row that lane l (0..15) of a half-warp holds: D/64 pieces of 4,
// contiguous over the lanes.
template <int D>
struct RowPiece {
  static constexpr int N = D / 16;
  __device__ __forceinline__ static int dim(int l, int i) { return (i >> 2) * 64 + l * 4 + (i & 3); }
  __device__ __forceinline__ static void load(const float* row, int l, float (&x)[N]) {
#pragma unroll
    for (int j = 0; j < N / 4; ++j) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(row + j * 64 + l * 4));
      x[4 * j] = v.x; x[4 * j + 1] = v.y; x[4 * j + 2] = v.z; x[4 * j + 3] = v.w;
    }
  }
};

template <int G, int D>
struct SimtSmem {
  PagedRunSmem run;
  union {
    float o[pds::NW][G][D];
    typename PagedJoin<pds::THREADS, G, D>::Smem join;
  };
  float m[pds::NW][G], l[pds::NW][G];
  int last;
};

template <int G, int D>
__global__ void __launch_bounds__(pds::THREADS, 1) paged_decode_simt_kernel(PagedDecodeArgs a) {
  using namespace pds;
  using Row = RowPiece<D>;
  constexpr int N = Row::N;
  __shared__ SimtSmem<G, D> sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, half = lane >> 4, l16 = lane & 15;
  const PagedRows rows = paged_rows(a);
  paged_begin();
  const int mine = paged_first_tiles(a);
  const PagedRun run = paged_run<THREADS>(a, sm.run, mine, SEG_COST, PARTS_PER_TILE);
  paged_empty_rows(a, tid, THREADS);
  const float sl2 = a.scale * 1.4426950408889634f;
  PagedWalk walk(run, SEG_COST);
  PagedPiece pc;
  while (walk.next(a, rows, pc)) {
    const PagedHead hd = paged_head(a, pc.row, pc.sub, HEADS);
    const int len = paged_len(a, hd.b);
    float q[G][N], acc[G][N], m[G], l[G];
#pragma unroll
    for (int h = 0; h < G; ++h) {
      const float* qr = static_cast<const float*>(a.q) + (size_t)hd.b * a.q_b + (size_t)(hd.h0 + (h < hd.nh ? h : 0)) * a.q_h;
      Row::load(qr, l16, q[h]);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        q[h][i] *= sl2;
        acc[h][i] = 0.f;
      }
      m[h] = -CUDART_INF_F;
      l[h] = 0.f;
    }
    for (int t = pc.a; t < pc.b; ++t) {
      // this half-warp's 8 consecutive keys lie in one page (pages hold at least 8 tokens)
      const int k0 = t * kPagedTile + (warp * 2 + half) * KPW;
      PagedSpan sp = paged_span(a, hd.b, hd.g, len, k0, KPW);
      sp.valid = paged_valid(a, sp);
      const size_t base = (size_t)max(sp.page, 0) * a.pool.page + (size_t)sp.in_page * a.pool.token +
                          (size_t)hd.g * a.pool.head;
      const float* kr = static_cast<const float*>(a.k) + base;
      const float* vr = static_cast<const float*>(a.v) + base;
#pragma unroll
      for (int u0 = 0; u0 < KPW; u0 += 4) {
        float kx[4][N], vx[4][N], s[4][G];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (u0 + u < sp.valid) {
            Row::load(kr + (size_t)(u0 + u) * a.pool.token, l16, kx[u]);
            Row::load(vr + (size_t)(u0 + u) * a.pool.token, l16, vx[u]);
          } else {
#pragma unroll
            for (int i = 0; i < N; ++i) kx[u][i] = vx[u][i] = 0.f;
          }
        }
        float mx[G];
#pragma unroll
        for (int h = 0; h < G; ++h) mx[h] = m[h];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int h = 0; h < G; ++h) {
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) x = fmaf(q[h][i], kx[u][i], x);
#pragma unroll
            for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            s[u][h] = u0 + u < sp.valid ? x : -CUDART_INF_F;
            mx[h] = fmaxf(mx[h], s[u][h]);
          }
#pragma unroll
        for (int h = 0; h < G; ++h) {
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 16));
          if (mx[h] > m[h]) {     // the same in the whole warp
            const float alpha = exp2f(m[h] - mx[h]);
            l[h] *= alpha;
#pragma unroll
            for (int i = 0; i < N; ++i) acc[h][i] *= alpha;
            m[h] = mx[h];
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float p = s[u][h] == -CUDART_INF_F ? 0.f : exp2f(s[u][h] - m[h]);
            l[h] += p;
#pragma unroll
            for (int i = 0; i < N; ++i) acc[h][i] = fmaf(p, vx[u][i], acc[h][i]);
          }
        }
      }
    }
    // ---- join the two half-warps, then the warps
#pragma unroll
    for (int h = 0; h < G; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 16);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float o = acc[h][i] + __shfl_xor_sync(0xffffffffu, acc[h][i], 16);
        if (half == 0) sm.o[warp][h][Row::dim(l16, i)] = o;
      }
      if (lane == 0) {
        sm.m[warp][h] = m[h];
        sm.l[warp][h] = l[h];
      }
    }
    __syncthreads();
    const bool whole = pc.a == 0 && pc.b == pc.nt;
    float* part = paged_part(a, blockIdx.x, run.t0 >= pc.seg_t ? 0 : 1);
    for (int e = tid; e < hd.nh * D; e += THREADS) {
      const int h = e / D, d = e - h * D;
      float mx = -CUDART_INF_F;
#pragma unroll
      for (int w = 0; w < NW; ++w) mx = fmaxf(mx, sm.m[w][h]);
      float L = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float al = sm.l[w][h] == 0.f ? 0.f : exp2f(sm.m[w][h] - mx);
        L = fmaf(al, sm.l[w][h], L);
        o = fmaf(al, sm.o[w][h][d], o);
      }
      o = L == 0.f ? 0.f : o / L;
      const float lse = L == 0.f ? -CUDART_INF_F : (mx + log2f(L)) * 0.6931471805599453f;
      if (whole) {
        const size_t bh = (size_t)hd.b * a.Hq + hd.h0 + h;
        paged_store(a, bh * D + d, o);
        if (d == 0 && a.out_lse) a.out_lse[bh] = lse;
      } else {
        part[h * D + d] = o;
        if (d == 0) part[kPagedHeads * D + h] = lse;
      }
    }
    __syncthreads();    // the parts are written, sm.o is free
    if (!whole) {
      const int c0 = run_owner(run, pc.seg_t), c1 = run_owner(run, pc.seg_t + pc.nt - 1);
      if (tid == 0) {
        const unsigned int old = atom_add_acq_rel_gpu(a.ws_count + c0, 1u);
        sm.last = old == (unsigned int)(c1 - c0);
        if (sm.last) atomicExch(a.ws_count + c0, 0u);    // zero again for the next call
      }
      __syncthreads();
      if (sm.last)
        paged_join<THREADS, G, D>(a, run, pc, hd, c0, c1, tid, sm.join, [] { __syncthreads(); });
    }
  }
}

template <int G>
static cudaError_t launch_simt(const PagedDecodeArgs& a, cudaStream_t st) {
  const int grid = min(num_sms(), kPagedMaxCtas);
  if (a.D == 64) return paged_launch(paged_decode_simt_kernel<G, 64>, grid, pds::THREADS, 0, st, a);
  return paged_launch(paged_decode_simt_kernel<G, 128>, grid, pds::THREADS, 0, st, a);
}

cudaError_t launch_paged_decode_simt(const PagedDecodeArgs& args, cudaStream_t st) {
  PagedDecodeArgs a = args;
  a.ngrp = (a.G + pds::HEADS - 1) / pds::HEADS;
  if (a.G == 1) return launch_simt<1>(a, st);
  if (a.G == 2) return launch_simt<2>(a, st);
  if (a.G <= 4) return launch_simt<4>(a, st);
  return launch_simt<8>(a, st);
}

static size_t part_bytes(int D) {
  return ((size_t)2 * kPagedMaxCtas * kPagedHeads * (D + 1) * sizeof(float) + 255) & ~size_t(255);
}
size_t paged_decode_workspace_bytes(int D) { return part_bytes(D) + ((kPagedMaxCtas * sizeof(unsigned int) + 255) & ~size_t(255)); }
void paged_decode_workspace_split(void* ws, int D, float** part, unsigned int** count) {
  *part = static_cast<float*>(ws);
  *count = reinterpret_cast<unsigned int*>(static_cast<uint8_t*>(ws) + part_bytes(D));
}

}  // namespace ra
