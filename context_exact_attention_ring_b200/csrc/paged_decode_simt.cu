// Paged decode on CUDA cores (float32 cache): one new token per sequence
// against the keys in its cache pages,
//   out_h = sum_j softmax_j(scale q_h . k_j) v_j,   lse_h = ln sum_j e^(scale q_h . k_j),
// in one pass over the keys with a running maximum and sum.  The tensor cores
// have no float32 product; every product and sum here is float32.
//
// A CTA of 16 warps takes the tiles of its run (paged_split.cuh) in units of 8
// keys to a group of D / 4 lanes, which share a key row (one contiguous load);
// a lane keeps 4 dims of the outputs of up to 8 heads in registers, as packed
// pairs.  K and V come by asynchronous copies into slots that the copying lane
// itself reads, so that no barrier is needed: the next unit's K while this
// one's V is used, its V during the next scores.  The 8 partial scores of a head
// are added up across the lanes by halving (4 + 2 + 1 exchanges leave a lane one
// key), so that a lane takes one maximum and one exponential per head; the
// weights return through shared memory as pairs.  Above two heads bound by the
// latency of a head's chain (exchanges, maximum, a branch, exponential) and of
// a piece's start, when the copies' pipeline is empty (with 5 heads issue slots
// are 44% busy, DRAM 50%), and by memory below.
// (Four keys at a time: 62 us for 400,000 rows of 5 heads of 64, eight: 57, with
// the runs weighed as now 48.)
#include <cuda_runtime.h>
#include <math_constants.h>

#include "kernels.h"
#include "paged_split.cuh"

namespace ra {

namespace pds {
constexpr int THREADS = 512;
constexpr int NW = THREADS / 32;
constexpr int HEADS = kPagedSimtHeads;  // query heads of a group, at most
// What a segment costs besides its tiles (queries, the empty pipeline, the warps' sums), in tiles; with 1
// the case of 5 heads took 57 us, with 2 and 3 it takes 48.
constexpr int SEG_COST = kPagedSimtSegCost;
constexpr int PARTS_PER_TILE = 20;     // parts joined in the time of a tile
}  // namespace pds

template <int G, int D>
struct SimtSmem {
  PagedRunSmem run;
  alignas(16) float q[G][D];
  float m[pds::NW][G], l[pds::NW][G];
  int last;
  // (weight, weight) per key of a lane group and head
  alignas(16) float2 p[pds::NW][128 / D][8][(G + 1) & ~1];
  union {
    uint4 kv[2][8][pds::THREADS];                         // K and V: 16 bytes of 8 keys for every lane
    float o[pds::NW][G][D];                               // between pieces
    typename PagedJoin<pds::THREADS, G, D>::Smem join;
  };
};

// 16 bytes to shared memory in the background; zeros (and no read) where !ok.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0)
               : "memory");
}

template <int G, int D>
__global__ void __launch_bounds__(pds::THREADS, 1) paged_decode_simt_kernel(PagedDecodeArgs a) {
  using namespace pds;
  constexpr int LPR = D / 4, RPW = 32 / LPR;      // lanes of a row, groups of a warp
  constexpr int UNIT = 8 * RPW;                   // keys a warp takes at a time, 8 a group (pages hold at least 8)
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SimtSmem<G, D>& sm = *reinterpret_cast<SimtSmem<G, D>*>(smem_raw);
  paged_begin();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, grp = lane / LPR, lr = lane % LPR;
  const PagedRows rows = paged_rows(a);
  const PagedRun run = paged_run<THREADS>(a, sm.run, paged_first_tiles(a), SEG_COST, PARTS_PER_TILE);
  paged_empty_rows(a, tid, THREADS);
  const float sl2 = a.scale * 1.4426950408889634f;
  // A lane takes its group's eight keys in the order u ^ mine, u = 0 .. 7.  A lane that differs from it
  // in one bit of `mine` then has the sum for the lane's place u at its own place u + 4 (2, 1): halving
  // needs no selection, and ends with key `mine` in place 0.
  const int mine = (lr & (LPR / 2) ? 4 : 0) + (lr & (LPR / 4) ? 2 : 0) + (lr & (LPR / 8) ? 1 : 0);
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
    const int nunits = (pc.b - pc.a) * (kPagedTile / UNIT);
    auto span = [&](int i) { return paged_span(a, hd.b, hd.g, len, pc.a * kPagedTile + i * UNIT + grp * 8, 8); };
    // 16 bytes of 8 keys of K (which 0) or V (1) to this lane's slots
    auto copy = [&](const PagedSpan& sp, int which) {
      const size_t base = (size_t)(sp.valid ? sp.page : 0) * a.pool.page + (size_t)sp.in_page * a.pool.token +
                          (size_t)hd.g * a.pool.head + 4 * lr;
      const float* row = static_cast<const float*>(which ? a.v : a.k) + base;
#pragma unroll
      for (int u = 0; u < 8; ++u, row += a.pool.token)      // rows of one page, valid or not
        copy16(&sm.kv[which][u][tid], row, u < sp.valid);
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
    PagedSpan cur, next;
    cur.valid = next.valid = 0;
    cur.page = next.page = cur.in_page = next.in_page = 0;
    if (warp < nunits) {
      cur = span(warp);
      cur.valid = paged_valid(a, cur);
      copy(cur, 0);
      commit();
      copy(cur, 1);
    }
    commit();
    if (warp + NW < nunits) next = span(warp + NW);
    for (int i = warp; i < nunits; i += NW) {
      const bool more = i + NW < nunits;
      next.valid = more ? paged_valid(a, next) : 0;
      asm volatile("cp.async.wait_group 1;" ::: "memory");      // K of this unit
      const bool valid = mine < cur.valid;
      {
        ulonglong2 kx[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) kx[u] = *reinterpret_cast<const ulonglong2*>(&sm.kv[0][u ^ mine][tid]);
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(&sm.q[h][4 * lr]);
          float s[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) s[u] = hsum2(ffma2(q.x, kx[u].x, fmul2(q.y, kx[u].y)));
          // keep the lower half of the places and send the sums of the upper, three times
#pragma unroll
          for (int u = 0; u < 4; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[4 + u], LPR / 2);
#pragma unroll
          for (int u = 0; u < 2; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[2 + u], LPR / 4);
          float x = s[0] + __shfl_xor_sync(0xffffffffu, s[1], LPR / 8);
#pragma unroll
          for (int o = LPR / 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
          if (!valid) x = -CUDART_INF_F;
          const float mx = warp_max_redux(x);
          if (mx > m[h]) {                          // the same in the whole warp
            const float alpha = ex2(m[h] - mx);
            const uint64_t al2 = pack2(alpha, alpha);
            l[h] *= alpha;
            acc[h][0] = fmul2(acc[h][0], al2);
            acc[h][1] = fmul2(acc[h][1], al2);
            m[h] = mx;
          }
          const float p = x == -CUDART_INF_F ? 0.f : ex2(x - m[h]);
          l[h] += p;                                // every key in LPR / 8 lanes
          if (lr % (LPR / 8) == 0) sm.p[warp][grp][mine][h] = make_float2(p, p);
        }
      }
      if (more) copy(next, 0);
      commit();
      asm volatile("cp.async.wait_group 1;" ::: "memory");      // V of this unit
      __syncwarp();
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const ulonglong2 vx = *reinterpret_cast<const ulonglong2*>(&sm.kv[1][u][tid]);
        const ulonglong2* pp = reinterpret_cast<const ulonglong2*>(sm.p[warp][grp][u]);
#pragma unroll
        for (int h = 0; h < G; h += 2) {
          const ulonglong2 w = pp[h / 2];
          acc[h][0] = ffma2(w.x, vx.x, acc[h][0]);
          acc[h][1] = ffma2(w.x, vx.y, acc[h][1]);
          if (h + 1 < G) {
            acc[h + 1 < G ? h + 1 : h][0] = ffma2(w.y, vx.x, acc[h + 1 < G ? h + 1 : h][0]);
            acc[h + 1 < G ? h + 1 : h][1] = ffma2(w.y, vx.y, acc[h + 1 < G ? h + 1 : h][1]);
          }
        }
      }
      __syncwarp();                                 // sm.p has been read
      if (more) copy(next, 1);
      commit();
      cur = next;
      if (i + 2 * NW < nunits) next = span(i + 2 * NW);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();                                // sm.kv has been read
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
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], LPR / 8);
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

// Workspace: the counters first, so that they stay in place (and zero) when calls of either head dimension
// use one workspace in turn, then the parts.
static constexpr size_t kCountBytes = (kPagedMaxCtas * sizeof(unsigned int) + 255) & ~size_t(255);
size_t paged_decode_workspace_bytes(int D) {
  return kCountBytes + (((size_t)2 * kPagedMaxCtas * kPagedHeads * (D + 1) * sizeof(float) + 255) & ~size_t(255));
}
void paged_decode_workspace_split(void* ws, float** part, unsigned int** count) {
  *count = static_cast<unsigned int*>(ws);
  *part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kCountBytes);
}

}  // namespace ra
