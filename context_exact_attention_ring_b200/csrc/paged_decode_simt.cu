// Paged decode on CUDA cores (float32 cache): one new token per sequence
// against the keys in its cache pages,
//   out_h = sum_j softmax_j(scale q_h . k_j) v_j,   lse_h = ln sum_j e^(scale q_h . k_j),
// in one pass over the keys with a running maximum and sum.  The tensor cores
// have no float32 product; every product and sum here is float32.
//
// A CTA of 16 warps takes the tiles of its run (paged_split.cuh), 8 keys a
// warp.  D / 4 lanes share a key row (one contiguous load), and each lane keeps
// 4 dims of the outputs of up to 8 heads in registers, as packed pairs.  Four keys go through at once: their partial scores are added up
// across the lanes by halving (2 + 1 exchanges leave a lane one key, the rest
// are plain), so that a lane ends with one score and takes one exponential per
// head, and the four weights return by shuffles.  Bound by memory for few heads and
// by instructions for many: about 55 per head and four keys of a warp.
#include <cuda_runtime.h>
#include <math_constants.h>

#include "kernels.h"
#include "paged_split.cuh"

namespace ra {

namespace pds {
constexpr int THREADS = 512;
constexpr int NW = THREADS / 32;
constexpr int KPW = kPagedTile / NW;   // keys of a tile a warp takes
constexpr int HEADS = 8;               // query heads of a group, at most
constexpr int SEG_COST = 1;            // what a segment costs besides its tiles, in tiles
constexpr int PARTS_PER_TILE = 10;     // parts joined in the time of a tile
static_assert(KPW == 8, "a warp's keys lie in one page (pages hold at least 8 tokens)");
}  // namespace pds

template <int G, int D>
struct SimtSmem {
  PagedRunSmem run;
  alignas(16) float q[G][D];
  float m[pds::NW][G], l[pds::NW][G];
  int last;
  union {
    float o[pds::NW][G][D];
    typename PagedJoin<pds::THREADS, G, D>::Smem join;
  };
};

template <int G, int D>
__global__ void __launch_bounds__(pds::THREADS, 1) paged_decode_simt_kernel(PagedDecodeArgs a) {
  using namespace pds;
  constexpr int LPR = D / 4, RPW = 32 / LPR;      // lanes of a row, rows a warp loads at once
  constexpr int NB = KPW / (4 * RPW);             // batches of 4 keys per group of lanes
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SimtSmem<G, D>& sm = *reinterpret_cast<SimtSmem<G, D>*>(smem_raw);
  paged_begin();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, grp = lane / LPR, lr = lane % LPR;
  const PagedRows rows = paged_rows(a);
  const PagedRun run = paged_run<THREADS>(a, sm.run, paged_first_tiles(a), SEG_COST, PARTS_PER_TILE);
  paged_empty_rows(a, tid, THREADS);
  const float sl2 = a.scale * 1.4426950408889634f;
  // after the exchanges a lane holds key `mine` of its group's four
  const bool b1 = lr & (LPR / 2), b0 = lr & (LPR / 4);
  const int mine = (b1 ? 2 : 0) + (b0 ? 1 : 0);
  PagedWalk walk(a, rows, run, SEG_COST);
  PagedPiece pc;
  while (walk.next(a, rows, pc)) {
    const PagedHead hd = paged_head(a, pc.row, pc.sub, HEADS);
    const int len = paged_len(a, hd.b);
    // the queries, scaled, in shared memory (free since the barriers of the piece before)
    for (int e = tid; e < G * D; e += THREADS) {
      const int h = e / D;
      sm.q[h][e - h * D] = h < hd.nh ? static_cast<const float*>(a.q)[(size_t)hd.b * a.q_b + (size_t)(hd.h0 + h) * a.q_h +
                                                                      e - h * D] * sl2
                                     : 0.f;
    }
    uint64_t acc[G][2];
    float m[G], l[G];
#pragma unroll
    for (int h = 0; h < G; ++h) {
      acc[h][0] = acc[h][1] = pack2(0.f, 0.f);
      m[h] = -CUDART_INF_F;
      l[h] = 0.f;
    }
    __syncthreads();
    auto span = [&](int t) { return paged_span(a, hd.b, hd.g, len, t * kPagedTile + warp * KPW, KPW); };
    PagedSpan next = span(pc.a);
    for (int t = pc.a; t < pc.b; ++t) {
      PagedSpan sp = next;
      if (t + 1 < pc.b) next = span(t + 1);
      sp.valid = paged_valid(a, sp);
      if (sp.valid == 0) continue;                // the same in the whole warp
      const size_t base = (size_t)sp.page * a.pool.page + (size_t)sp.in_page * a.pool.token +
                          (size_t)hd.g * a.pool.head + 4 * lr;
      const float* kr = static_cast<const float*>(a.k) + base;
      const float* vr = static_cast<const float*>(a.v) + base;
#pragma unroll 1
      for (int n = 0; n < NB; ++n) {
        ulonglong2 kx[4], vx[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int key = (n * 4 + u) * RPW + grp;
          kx[u] = vx[u] = make_ulonglong2(0ull, 0ull);
          if (key < sp.valid) {
            kx[u] = __ldg(reinterpret_cast<const ulonglong2*>(kr + (size_t)key * a.pool.token));
            vx[u] = __ldg(reinterpret_cast<const ulonglong2*>(vr + (size_t)key * a.pool.token));
          }
        }
        const bool valid = (n * 4 + mine) * RPW + grp < sp.valid;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(&sm.q[h][4 * lr]);
          float s[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) s[u] = hsum2(ffma2(q.x, kx[u].x, fmul2(q.y, kx[u].y)));
          // keep two keys and send the others' sums, then one
          float s0 = b1 ? s[2] : s[0], s1 = b1 ? s[3] : s[1];
          s0 += __shfl_xor_sync(0xffffffffu, b1 ? s[0] : s[2], LPR / 2);
          s1 += __shfl_xor_sync(0xffffffffu, b1 ? s[1] : s[3], LPR / 2);
          float x = b0 ? s1 : s0;
          x += __shfl_xor_sync(0xffffffffu, b0 ? s0 : s1, LPR / 4);
#pragma unroll
          for (int o = LPR / 8; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
          if (!valid) x = -CUDART_INF_F;
          const float mx = warp_max_redux(x);
          if (mx > m[h]) {                        // the same in the whole warp
            const float alpha = exp2f(m[h] - mx);
            const uint64_t al2 = pack2(alpha, alpha);
            l[h] *= alpha;
            acc[h][0] = fmul2(acc[h][0], al2);
            acc[h][1] = fmul2(acc[h][1], al2);
            m[h] = mx;
          }
          const float p = x == -CUDART_INF_F ? 0.f : exp2f(x - m[h]);
          l[h] += p;                              // every key in LPR / 4 lanes
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int src = grp * LPR + (u & 2 ? LPR / 2 : 0) + (u & 1 ? LPR / 4 : 0);
            const float pu = __shfl_sync(0xffffffffu, p, src);
            const uint64_t p2 = pack2(pu, pu);
            acc[h][0] = ffma2(p2, vx[u].x, acc[h][0]);
            acc[h][1] = ffma2(p2, vx[u].y, acc[h][1]);
          }
        }
      }
    }
    // ---- the groups of lanes, then the warps
#pragma unroll
    for (int h = 0; h < G; ++h) {
      float4 o;
      unpack2(acc[h][0], o.x, o.y);
      unpack2(acc[h][1], o.z, o.w);
      if constexpr (RPW == 2) {
        o.x += __shfl_xor_sync(0xffffffffu, o.x, 16);
        o.y += __shfl_xor_sync(0xffffffffu, o.y, 16);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, 16);
        o.w += __shfl_xor_sync(0xffffffffu, o.w, 16);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 16);
      }
      // one lane of each key
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], LPR / 2);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], LPR / 4);
      if (grp == 0) *reinterpret_cast<float4*>(&sm.o[warp][h][4 * lr]) = o;
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
      if (sm.last) paged_join<THREADS, G, D>(a, run, pc, hd, c0, c1, tid, sm.join, [] { __syncthreads(); });
    }
  }
}

template <int G, int D>
static cudaError_t launch_simt_gd(const PagedDecodeArgs& a, cudaStream_t st) {
  auto kern = paged_decode_simt_kernel<G, D>;
  const cudaError_t e = paged_raise_smem<(int)sizeof(SimtSmem<G, D>)>(kern);
  if (e != cudaSuccess) return e;
  return paged_launch(kern, min(num_sms(), kPagedMaxCtas), pds::THREADS, sizeof(SimtSmem<G, D>), st, a);
}
template <int G>
static cudaError_t launch_simt(const PagedDecodeArgs& a, cudaStream_t st) {
  return a.D == 64 ? launch_simt_gd<G, 64>(a, st) : launch_simt_gd<G, 128>(a, st);
}

cudaError_t launch_paged_decode_simt(const PagedDecodeArgs& args, cudaStream_t st) {
  PagedDecodeArgs a = args;
  a.ngrp = (a.G + pds::HEADS - 1) / pds::HEADS;
  switch (a.G) {
    case 1: return launch_simt<1>(a, st);
    case 2: return launch_simt<2>(a, st);
    case 3: return launch_simt<3>(a, st);
    case 4: return launch_simt<4>(a, st);
    case 5: return launch_simt<5>(a, st);
    case 6: return launch_simt<6>(a, st);
    case 7: return launch_simt<7>(a, st);
    default: return launch_simt<8>(a, st);
  }
}

static size_t part_bytes(int D) {
  return ((size_t)2 * kPagedMaxCtas * kPagedHeads * (D + 1) * sizeof(float) + 255) & ~size_t(255);
}
size_t paged_decode_workspace_bytes(int D) {
  return part_bytes(D) + ((kPagedMaxCtas * sizeof(unsigned int) + 255) & ~size_t(255));
}
void paged_decode_workspace_split(void* ws, int D, float** part, unsigned int** count) {
  *part = static_cast<float*>(ws);
  *count = reinterpret_cast<unsigned int*>(static_cast<uint8_t*>(ws) + part_bytes(D));
}

}  // namespace ra
