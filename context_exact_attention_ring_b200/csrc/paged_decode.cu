// Paged decode on the tensor cores (bf16 cache): one new token per sequence
// against the keys in its cache pages, in one pass with a running maximum and
// sum, split over the keys and joined in the same launch (paged_split.cuh).
//
// The query heads of a kv head share every K/V row, so a 128-key tile is a
// pair of small tcgen05 products, heads padded to 16 columns:
//   S^T = K Q^T       M = 128 keys, N = 16 heads, K = D   (K, Q K-major)
//   O^T += V^T P^T    M = 128 dims, N = 2 x 8 or 2 x 16, K = 128 keys
// N = 16 is the narrowest product, so 8 heads leave half of its columns
// empty: the weights go in as two bf16 terms, p = hi + lo with |p - hi - lo|
// <= 2^-16 p, in columns of their own, for the price of the second
// shared-memory store.  Every FOLD tiles O^T is added to a sum beside it in
// tensor memory.  The float32 output is off by 2e-6 to 4e-6 of itself.
//
// Bound by HBM: a tile is 64 KB at D = 128 against 2 x 128 x 16 x D products
// (6 sequences of 64k to 128k keys, 32/8 heads of 128: 346 us, 6.7 TB/s; 64 ragged
// ones of 64 to 16,000: 103 us, 6.0 TB/s; one of 77 keys: 5.9 us).
// One CTA per SM; warp roles:
//   warps 0-3  softmax: thread t owns tensor-memory lane t (key row t of S^T,
//              dim t of O^T);
//   warps 4, 6 producers of K (and Q) and of V: lane i owns page slot i of a
//              tile (a tile holds 128 / page_size pages, or is part of one),
//              looks its page up one tile ahead and issues its page's TMA
//              boxes into a ring of stages.  Issuing a box takes 60-80 cycles
//              (120 if one lane does it for all), and a tile of 16-token
//              pages is 32 boxes in the 2700 cycles its bytes take: hence two
//              warps.  The V producer also leaves each slot's number of valid
//              keys (its stage is not refilled before the softmax is done with
//              the tile; K's is free as soon as S^T is);
//   warp 5     MMA issuer and tensor-memory owner.  Tiles follow each other
//              across segments without a drain: S^T(t+1) is issued before
//              O^T(t), and Q, O^T and the weights have two buffers.
// A key that is not valid (past the length, or in an absent page) has weight 0
// and its V row is zeroed in shared memory, whatever the page held there.
// Every wait is bounded.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <type_traits>

#include "kernels.h"
#include "paged.h"
#include "paged_split.cuh"
#include "ptx.cuh"

namespace ra {

namespace pdt {
constexpr int NQ = 16;                      // heads per CTA, padded
constexpr int SLAB = kPagedTile * 128;      // 128 rows x 64 columns of bf16 (16 KB)
constexpr int QSLAB = NQ * 128;
constexpr int CT = 128;                     // softmax threads
constexpr int THREADS = CT + 96;
constexpr uint32_t TMEM_COLS = 128;         // S^T 2 x 16, O^T 2 x (16 or 32), folded sums of up to 16 heads
constexpr float LAZY = 8.f;                 // log2 of the growth tolerated before the base moves
// K/V stages: what shared memory holds (D = 64, 56 sequences of 16,000 keys: 404 us with 3, 395 with 5).
template <int DH>
constexpr int NST = DH == 64 ? 5 : 3;
constexpr int MAX_SLOTS = kPagedTile / 8;   // page slots of a tile
// What a segment costs besides its tiles, in tiles: its result's sums, divisions and stores grow with the
// heads (64 ragged sequences with 16 heads to a kv head: 129 us with 1, 111 with 2; with 4 heads 103 and 103,
// 128 shorter ones 54 and 57).
template <int G>
constexpr int SEG_COST = paged_seg_cost(G);
constexpr int PARTS_PER_TILE = 20;          // parts joined in the time of a tile
// Tiles added up in the products' accumulator before it is folded into a float32 sum that rounds: the tensor
// cores drop what does not fit, always towards zero.  1M keys to a CTA: outputs off by 9e-4 of themselves (6.5e-3
// with values of one sign) without folding, 1e-5 with 64 tiles, 5e-6 with 32, 3e-6 with 16 (4e-6 with values of
// one sign), about as with few keys; the times are the same (6 sequences of 64k to 128k keys).
constexpr int FOLD = 16;
}  // namespace pdt

template <int G, int DH>
struct PagedSmem {
  static constexpr int GP = G <= 8 ? 8 : 16;  // weight columns of a term
  static constexpr int NP = 2 * GP;           // weight columns: hi, lo
  static constexpr int PSLAB = NP * 128;      // 64 keys of all weight columns
  static constexpr int NST = pdt::NST<DH>;
  alignas(1024) uint8_t kv[NST][2][(DH / 64) * pdt::SLAB];
  // D = 64: the upper 64 of the M = 128 dims of O^T, common to all stages
  alignas(1024) uint8_t zero[DH == 64 ? pdt::SLAB : 1];
  alignas(1024) uint8_t q[2][2 * pdt::QSLAB];
  alignas(1024) uint8_t pt[2][2 * PSLAB];
  int nvalid[NST][pdt::MAX_SLOTS];       // valid keys per page slot of a V stage
  alignas(16) float red[2][GP][4];            // the warps' maxima, by tile parity
  alignas(16) float suml[2][GP][4];           // the warps' sums, by piece parity
  float base[2][GP];                          // final bases
  alignas(16) typename PagedJoin<pdt::CT, G, DH>::Smem join;
  // mbarriers
  alignas(8) uint64_t k_full[NST], k_empty[NST], v_full[NST], v_empty[NST];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_done[2], o_full[2], o_free[2], teardown;
  PagedRunSmem run;
  uint32_t tmem_base;
  int is_last, abort_flag;
};

struct PagedMaps {
  int head_outer;     // the pools' head stride is the larger: box order (D, token, head, page)
  int q_rows;         // rows of a query box
};

__host__ __device__ constexpr uint32_t paged_idesc(int N, bool a_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}

// N consecutive 32-bit columns of this warp's lanes, N = 1, 2, 4, 8, 16
template <int N>
__device__ __forceinline__ void paged_tmem_ld(uint32_t t, float (&v)[N]) {
  uint32_t r[N];
  if constexpr (N == 1)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r[0]) : "r"(t));
  else if constexpr (N == 2)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(t));
  else if constexpr (N == 4)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(t));
  else if constexpr (N == 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(t));
  else
    tmem_ld16(t, r);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}
template <int N>
__device__ __forceinline__ void paged_tmem_st(uint32_t t, const float (&v)[N]) {
  uint32_t r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = __float_as_uint(v[i]);
  if constexpr (N == 1)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(t), "r"(r[0]) : "memory");
  else if constexpr (N == 2)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};" ::"r"(t), "r"(r[0]), "r"(r[1]) : "memory");
  else if constexpr (N == 4)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(t), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]) : "memory");
  else if constexpr (N == 8)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
  else
    tmem_st16(t, r);
}

// The sum of a product's two terms.  An infinite value times a weight's second
// term, 0 or of either sign, is no part of it.
__device__ __forceinline__ float paged_terms(float hi, float lo) { return fabsf(hi) < CUDART_INF_F ? hi + lo : hi; }

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

template <int G, int DH>
__global__ void __launch_bounds__(pdt::THREADS, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, PagedDecodeArgs a, PagedMaps maps) {
  using namespace pdt;
  using Smem = PagedSmem<G, DH>;
  constexpr int GP = Smem::GP, NP = Smem::NP, PSLAB = Smem::PSLAB, NST = Smem::NST;
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm.abort_flag;
  unsigned int* err = a.err;
  const PagedRows rows = paged_rows(a);
  const int psn_log2 = min(a.ps_log2, 7), psn = 1 << psn_log2;   // rows of a page slot

  paged_begin();
  // few rows: every warp plans by itself, and the producers start while the others set up
  const bool few = rows.R <= 32;
  const int mine = !few ? paged_first_tiles(a) : lane < rows.R ? paged_tiles(a, lane) : 0;   // on its way meanwhile
  if (threadIdx.x == 4 * 32) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
  }
  if (threadIdx.x == 6 * 32) tma_prefetch_desc(&tmV);
  if (warp == 0) {
    // a barrier per lane at a time; those the softmax threads arrive on count all of them
    for (uint32_t bar = smem_u32(&sm.k_full[0]) + 8 * lane; bar <= smem_u32(&sm.teardown); bar += 8 * 32) {
      const bool by_all = (bar >= smem_u32(&sm.p_full[0]) && bar < smem_u32(&sm.o_done[0])) ||
                          (bar >= smem_u32(&sm.o_free[0]) && bar < smem_u32(&sm.teardown));
      mbar_init(bar, by_all ? CT : 1);
    }
    if (lane == 0) sm.abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  const PagedRun run = few ? paged_run_warp(a, mine, SEG_COST<G>, PARTS_PER_TILE)
                           : paged_run<THREADS>(a, sm.run, mine, SEG_COST<G>, PARTS_PER_TILE);
  uint32_t tmem = 0;
  if (warp != 4 && warp != 6) {
    // the query rows past the box and all weight columns are zero (the copies write neither), and so are
    // the dims past D = 64
    constexpr int NT = THREADS - 64;
    const int tid = warp == 5 ? CT + lane : threadIdx.x;
    uint4* z = reinterpret_cast<uint4*>(&sm.q[0][0]);
    for (int i = tid; i < (int)sizeof(sm.q) / 16; i += NT)
      if ((i >> 3) % NQ >= maps.q_rows) z[i] = make_uint4(0u, 0u, 0u, 0u);
    z = reinterpret_cast<uint4*>(&sm.pt[0][0]);
    for (int i = tid; i < (int)sizeof(sm.pt) / 16; i += NT) z[i] = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (DH == 64) {
      z = reinterpret_cast<uint4*>(sm.zero);
      for (int i = tid; i < SLAB / 16; i += NT) z[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
    if (warp == 5) {
      tmem_alloc(smem_u32(&sm.tmem_base), TMEM_COLS);
      tmem_relinquish();
    }
    tc_fence_before();
    named_bar_sync(2, NT);
    tc_fence_after();
    tmem = sm.tmem_base;
  }

  if (warp == 4 || warp == 6) {
    // ------------------------------------------------------------ producers
    const bool is_k = warp == 4;
    const CUtensorMap* tmKV = is_k ? &tmK : &tmV;
    uint64_t* full = is_k ? sm.k_full : sm.v_full;
    uint64_t* empty = is_k ? sm.k_empty : sm.v_empty;
    const uint64_t pol_kv = l2_policy_evict_first(), pol_q = l2_policy_evict_last();
    const int nslots = kPagedTile >> psn_log2;
    PagedWalk walk(a, rows, run, SEG_COST<G>);
    PagedPiece pc;
    PagedHead hd{};
    int len = 0;
    auto span = [&](int j) {
      PagedSpan s;
      s.valid = 0;
      s.page = s.in_page = 0;
      if (lane < nslots) s = paged_span(a, hd.b, hd.g, len, j * kPagedTile + (lane << psn_log2), psn);
      return s;
    };
    // the tile after the one being loaded: its piece, and its pages (looked up one tile ahead)
    int j = 0;
    bool more = walk.next(a, rows, pc), starts = true;
    PagedSpan next;
    if (more) {
      hd = paged_head(a, pc.row, pc.sub, NQ);
      len = paged_len(a, hd.b);
      j = pc.a;
      next = span(j);
    }
    uint32_t cnt = 0, nq = 0;
    while (more) {
      PagedSpan cur = next;
      const int g = hd.g, h0 = hd.h0, b = hd.b;
      const bool new_q = starts;
      starts = ++j == pc.b;
      if (starts) {
        more = walk.next(a, rows, pc);
        if (more) {
          hd = paged_head(a, pc.row, pc.sub, NQ);
          len = paged_len(a, hd.b);
          j = pc.a;
        }
      }
      if (more) next = span(j);
      if (new_q && is_k) {
        const int qb = nq & 1;
        bool ok = nq < 2 || mbar_wait(smem_u32(&sm.q_empty[qb]), ((nq >> 1) - 1) & 1u, abort_flag, kWaitQEmpty, err);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (elect_one()) {
          const uint32_t qf = smem_u32(&sm.q_full[qb]);
          mbar_arrive_expect_tx(qf, (uint32_t)maps.q_rows * DH * 2);
          for (int sl = 0; sl < DH / 64; ++sl)
            tma_load_4d(smem_u32(sm.q[qb]) + sl * QSLAB, &tmQ, qf, sl * 64, h0, b, 0, pol_q);
        }
        ++nq;
      }
      const int s = cnt % NST;
      const bool ok = mbar_wait(smem_u32(&empty[s]), ((cnt / NST) & 1u) ^ 1u, abort_flag, kWaitDecodeEmpty, err);
      if (!__all_sync(0xffffffffu, ok)) break;
      cur.valid = paged_valid(a, cur);
      const uint32_t live = __ballot_sync(0xffffffffu, cur.valid > 0);
      if (!is_k && lane < MAX_SLOTS) sm.nvalid[s][lane] = cur.valid;
      __syncwarp();
      const uint32_t fb = smem_u32(&full[s]), dst = smem_u32(sm.kv[s][is_k ? 0 : 1]);
      if (lane == 0) mbar_arrive_expect_tx(fb, (uint32_t)__popc(live) * (uint32_t)(DH * 2) << psn_log2);
      __syncwarp();
      if (cur.valid > 0) {
        const int c1 = maps.head_outer ? cur.in_page : g, c2 = maps.head_outer ? g : cur.in_page;
        const uint32_t at = dst + ((uint32_t)lane << (psn_log2 + 7));
#pragma unroll
        for (int sl = 0; sl < DH / 64; ++sl) tma_load_4d(at + sl * SLAB, tmKV, fb, sl * 64, c1, c2, cur.page, pol_kv);
      }
      ++cnt;
    }
    __syncwarp();
    // do not leave while copies are still landing in shared memory
    if (lane == 0) {
      for (uint32_t c = (cnt > (uint32_t)NST ? cnt - NST : 0); c < cnt; ++c)
        mbar_wait(smem_u32(&full[c % NST]), (c / NST) & 1u, nullptr, kWaitTeardown, err);
      for (uint32_t c = (nq > 2u ? nq - 2u : 0u); c < nq; ++c)
        mbar_wait(smem_u32(&sm.q_full[c & 1]), (c >> 1) & 1u, nullptr, kWaitTeardown, err);
    }
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks, waits and computes addresses, so that these stay warp-uniform; one elected lane
    // (the same one every time) issues a product's instructions and the commits that track them.  With one
    // lane doing everything a tile took 2,150 cycles to issue, more than its bytes take at D = 64.
    constexpr uint32_t idS = paged_idesc(NQ, false), idPV = paged_idesc(NP, true);
    constexpr uint32_t HI = (1024u >> 4) | (1u << 14) | (2u << 29);    // stride 1024, version 1, 128-byte swizzle
    auto desc = [](uint32_t addr, uint32_t lbo) { return (addr >> 4) | (lbo >> 4) << 16; };
    PagedWalk walk(a, rows, run, SEG_COST<G>);
    PagedPiece pc;
    uint32_t t = 0, nu = 0;
    bool ok = true;
    bool prev_first = false, prev_last = false;
    uint32_t prev_u = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity, unsigned int site) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, abort_flag, site, err));
    };
    // O^T += V^T P^T of tile tt
    auto pv = [&](uint32_t tt) -> bool {
      const uint32_t s = tt % NST, pb = tt & 1u, ob = prev_u & 1u;
      // the softmax had V before it gave its weights
      if (!wait(&sm.p_full[pb], (tt >> 1) & 1u, kWaitPFull)) return false;
      if (prev_first && prev_u >= 2 && !wait(&sm.o_free[ob], ((prev_u >> 1) - 1) & 1u, kWaitOFinal)) return false;
      tc_fence_after();
      // the second 64 dims lie one slab further, or in the common zeros
      const uint32_t v0 = smem_u32(sm.kv[s][1]);
      const uint32_t vd = desc(v0, DH == 128 ? SLAB : smem_u32(sm.zero) - v0), pd = desc(smem_u32(sm.pt[pb]), 16);
      const uint32_t tO = tmem + 32 + ob * NP;
      if (elect_one()) {
        if (prev_first)
          mma_ss_lo_first(tO, vd, pd, HI, idPV);
        else
          mma_ss_lo(tO, vd, pd, HI, idPV);
#pragma unroll
        for (int k = 1; k < kPagedTile / 16; ++k)
          mma_ss_lo(tO, vd + ((k * 16 * 128) >> 4), pd + (((k >> 2) * PSLAB + (k & 3) * 32) >> 4), HI, idPV);
        mma_commit(smem_u32(&sm.o_done[pb]));
        mma_commit(smem_u32(&sm.v_empty[s]));
        if (prev_last) mma_commit(smem_u32(&sm.o_full[ob]));
      }
      __syncwarp();
      return true;
    };
    PagedPiece nxt;
    bool more = walk.next(a, rows, nxt);
    while (ok && more) {
      pc = nxt;
      more = walk.next(a, rows, nxt);      // while the piece's first copies are on their way
      const int qb = nu & 1;
      if (!wait(&sm.q_full[qb], (nu >> 1) & 1u, kWaitQFull)) {
        ok = false;
        break;
      }
      const uint32_t qd = desc(smem_u32(sm.q[qb]), 16);
      for (int j = pc.a; j < pc.b && ok; ++j) {
        const uint32_t s = t % NST, sb = t & 1u;
        // the scores' buffer is free: the softmax gave the weights of tile t - 2, which O^T(t - 2) waited for
        if (!wait(&sm.k_full[s], (t / NST) & 1u, kWaitDecodeFull)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t kd = desc(smem_u32(sm.kv[s][0]), 16), tS = tmem + 16 * sb;
        if (elect_one()) {
          mma_ss_lo_first(tS, kd, qd, HI, idS);
#pragma unroll
          for (int k = 1; k < DH / 16; ++k)
            mma_ss_lo(tS, kd + (((k >> 2) * SLAB + (k & 3) * 32) >> 4), qd + (((k >> 2) * QSLAB + (k & 3) * 32) >> 4), HI,
                      idS);
          mma_commit(smem_u32(&sm.s_full[sb]));
          mma_commit(smem_u32(&sm.k_empty[s]));
          if (j == pc.b - 1) mma_commit(smem_u32(&sm.q_empty[qb]));
        }
        __syncwarp();
        if (t > 0) ok = pv(t - 1);
        prev_first = j == pc.a;
        prev_last = j == pc.b - 1;
        prev_u = nu;
        ++t;
      }
      ++nu;
    }
    if (ok && t > 0) pv(t - 1);
    // every product issued so far must be complete before tensor memory is freed
    if (elect_one()) mma_commit(smem_u32(&sm.teardown));
    __syncwarp();
    mbar_wait(smem_u32(&sm.teardown), 0, nullptr, kWaitTeardown, err);
  } else {
    // ------------------------------------------------------------ softmax
    const int row = threadIdx.x;                              // key row of S^T, dim of O^T
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const float sl2 = a.scale * 1.4426950408889634f;
    const int slot = row >> psn_log2, in_slot = row & (psn - 1);
    // this thread's key in the weight operand: 16-byte chunk kc (XOR row) of 64-key slab row >> 6
    const uint32_t pt_base = (uint32_t)((row >> 6) * PSLAB + (row & 7) * 2);
    const int kc = (row & 63) >> 3;
    paged_empty_rows(a, row, CT);
    // the piece whose products are all issued, to be finished while the next one's run
    PagedPiece fpc{};
    PagedHead fhd{};
    float fl[G];
    uint32_t fu = 0;
    // sums folded so far of the present piece and of the one to be finished: whether there are any
    bool folded = false, ffolded = false;
    const uint32_t tA = tmem + lane_off + 32 + 2 * NP;
    auto finish = [&]() -> bool {
      const uint32_t ob = fu & 1u;
      const bool fin = mbar_wait(smem_u32(&sm.o_full[ob]), (fu >> 1) & 1u, abort_flag, kWaitOFinal, err);
      __syncwarp();
      tc_fence_after();
      float o[G], olo[G];
      const uint32_t tO = tmem + lane_off + 32 + ob * NP;
      paged_tmem_ld<G>(tO, o);
      paged_tmem_ld<G>(tO + GP, olo);
      tmem_wait_ld();
#pragma unroll
      for (int h = 0; h < G; ++h) o[h] = paged_terms(o[h], olo[h]);
      if (ffolded) {
        paged_tmem_ld<G>(tA, olo);
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < G; ++h) o[h] += olo[h];
      }
      tc_fence_before();
      mbar_arrive(smem_u32(&sm.o_free[ob]));
      ++fu;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        float s = fl[h];
#pragma unroll
        for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        if (lane == 0) sm.suml[ob][h][warp] = s;
      }
      if (named_bar_any(1, CT, !fin)) return false;
      const bool whole = fpc.a == 0 && fpc.b == fpc.nt;
      float* part = paged_part(a, blockIdx.x, run.t0 >= fpc.seg_t ? 0 : 1);
      const size_t bh0 = (size_t)fhd.b * a.Hq + fhd.h0;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        if (h >= fhd.nh) continue;
        const float4 r = *reinterpret_cast<const float4*>(sm.suml[ob][h]);
        const float L = (r.x + r.y) + (r.z + r.w);
        const float od = L == 0.f ? 0.f : __fdividef(o[h], L);
        if (row >= DH) continue;      // D = 64: the upper half of O^T is padding
        if (whole)
          paged_store(a, (bh0 + h) * DH + row, od);
        else
          part[h * DH + row] = od;
      }
      if (row < fhd.nh) {
        const float4 r = *reinterpret_cast<const float4*>(sm.suml[ob][row]);
        const float L = (r.x + r.y) + (r.z + r.w);
        const float lse = L == 0.f ? -CUDART_INF_F : (sm.base[ob][row] + log2f(L)) * 0.6931471805599453f;
        if (!whole)
          part[kPagedHeads * DH + row] = lse;
        else if (a.out_lse)
          a.out_lse[bh0 + row] = lse;
      }
      if (!whole) {
        const int c0 = run_owner(run, fpc.seg_t), c1 = run_owner(run, fpc.seg_t + fpc.nt - 1);
        named_bar_sync(1, CT);      // the part is written
        if (row == 0) {
          const unsigned int old = atom_add_acq_rel_gpu(a.ws_count + c0, 1u);
          sm.is_last = old == (unsigned int)(c1 - c0);
          if (sm.is_last) atomicExch(a.ws_count + c0, 0u);    // zero again for the next call
        }
        named_bar_sync(1, CT);
        if (sm.is_last)
          paged_join<CT, G, DH>(a, run, fpc, fhd, c0, c1, row, sm.join, [] { named_bar_sync(1, CT); });
      }
      return true;
    };

    PagedWalk walk(a, rows, run, SEG_COST<G>);
    PagedPiece pc;
    uint32_t t = 0, nu = 0;
    PagedPiece nxt;
    bool ok = true, more = walk.next(a, rows, nxt);
    while (ok && more) {
      pc = nxt;
      float m[G], l[G];      // per head: base (the same in every thread), this thread's sum
#pragma unroll
      for (int h = 0; h < G; ++h) {
        m[h] = -CUDART_INF_F;
        l[h] = 0.f;
      }
      for (int j = pc.a; j < pc.b; ++j, ++t) {
        const uint32_t sb = t & 1u, st = t % NST;
        // the tile's V and valid counts, and its scores; these were committed after O^T(t - 2), so that
        // its weight buffer is free as well
        bool good = mbar_wait(smem_u32(&sm.v_full[st]), (t / NST) & 1u, abort_flag, kWaitDecodeFull, err);
        if (good) good = mbar_wait(smem_u32(&sm.s_full[sb]), (t >> 1) & 1u, abort_flag, kWaitSFull, err);
        __syncwarp();
        tc_fence_after();
        float xs[G];
        paged_tmem_ld<G>(tmem + lane_off + 16 * sb, xs);
        tmem_wait_ld();
        const bool valid = in_slot < sm.nvalid[st][slot];
        if (!valid) {
          // neighbouring rows start at different 16-byte columns: 4 rows a wavefront, not 1
          uint4* vr = reinterpret_cast<uint4*>(sm.kv[st][1] + row * 128);
#pragma unroll
          for (int sl = 0; sl < DH / 64; ++sl)
#pragma unroll
            for (int c = 0; c < 8; ++c) vr[sl * (SLAB / 16) + ((c + row) & 7)] = make_uint4(0u, 0u, 0u, 0u);
        }
        __syncwarp();
        bool exceed = false;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          xs[h] = valid ? xs[h] * sl2 : -CUDART_INF_F;
          exceed |= xs[h] > m[h] + LAZY;
        }
        // a piece's first tile always sets the bases; later ones only where a score exceeds one
        if (j == pc.a || named_bar_any(1, CT, exceed || !good)) {
          const int rb = t & 1;
#pragma unroll
          for (int h = 0; h < G; ++h) {
            const float mw = warp_max_redux(xs[h]);
            if (lane == 0) sm.red[rb][h][warp] = mw;
          }
          if (named_bar_any(1, CT, !good)) {
            ok = false;
            break;
          }
          float alpha[G];
          bool moved = false;
#pragma unroll
          for (int h = 0; h < G; ++h) {
            const float4 r = *reinterpret_cast<const float4*>(sm.red[rb][h]);
            const float mt = fmaxf(fmaxf(r.x, r.y), fmaxf(r.z, r.w));
            alpha[h] = 1.f;
            if (mt > m[h] + LAZY) {
              alpha[h] = m[h] == -CUDART_INF_F ? 0.f : ex2(m[h] - mt);
              m[h] = mt;
              moved = true;
            }
            l[h] *= alpha[h];
          }
          if (j > pc.a && moved) {
            // rescale O^T once it holds the piece's earlier tiles; the same decision in every thread
            const uint32_t tp = t - 1;
            good = mbar_wait(smem_u32(&sm.o_done[tp & 1u]), (tp >> 1) & 1u, abort_flag, kWaitPFull, err);
            __syncwarp();
            tc_fence_after();
            const uint32_t tO = tmem + lane_off + 32 + (nu & 1u) * NP;
            float o[G];
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              paged_tmem_ld<G>(tO + part * GP, o);
              tmem_wait_ld();
#pragma unroll
              for (int h = 0; h < G; ++h) o[h] *= alpha[h];
              paged_tmem_st<G>(tO + part * GP, o);
            }
            if (folded) {
              paged_tmem_ld<G>(tA, o);
              tmem_wait_ld();
#pragma unroll
              for (int h = 0; h < G; ++h) o[h] *= alpha[h];
              paged_tmem_st<G>(tA, o);
            }
            tmem_wait_st();
            if (named_bar_any(1, CT, !good)) {
              ok = false;
              break;
            }
          }
        }
        if (j > pc.a && (j - pc.a) % FOLD == 0) {      // the same in every thread
          const uint32_t tp = t - 1;
          good = mbar_wait(smem_u32(&sm.o_done[tp & 1u]), (tp >> 1) & 1u, abort_flag, kWaitPFull, err);
          __syncwarp();
          tc_fence_after();
          const uint32_t tO = tmem + lane_off + 32 + (nu & 1u) * NP;
          constexpr int C = G < 4 ? G : 4;
#pragma unroll
          for (int h0 = 0; h0 < G; h0 += C) {
            float x[C], y[C];
            paged_tmem_ld<C>(tO + h0, x);
            paged_tmem_ld<C>(tO + GP + h0, y);
            tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < C; ++h) x[h] = paged_terms(x[h], y[h]);
            if (folded) {
              paged_tmem_ld<C>(tA + h0, y);
              tmem_wait_ld();
#pragma unroll
              for (int h = 0; h < C; ++h) x[h] += y[h];
            }
            paged_tmem_st<C>(tA + h0, x);
#pragma unroll
            for (int h = 0; h < C; ++h) x[h] = 0.f;
            paged_tmem_st<C>(tO + h0, x);
            paged_tmem_st<C>(tO + GP + h0, x);
          }
          tmem_wait_st();
          folded = true;
          if (named_bar_any(1, CT, !good)) {
            ok = false;
            break;
          }
        }
        // weights against the base, as two bf16 terms, for the tensor cores
        uint8_t* ptb = sm.pt[sb] + pt_base;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float pw = xs[h] == -CUDART_INF_F ? 0.f : ex2(xs[h] - m[h]);
          l[h] += pw;
          const uint32_t hi = pack_bf16x2(pw, 0.f) & 0xffffu;
          const uint32_t lo = pack_bf16x2(pw - __uint_as_float(hi << 16), 0.f);
          constexpr int lo_off = (GP >> 3) * 1024;     // GP rows further down
          uint8_t* at = ptb + (h >> 3) * 1024 + (h & 7) * 128 + ((kc ^ (h & 7)) << 4);
          *reinterpret_cast<uint16_t*>(at) = (uint16_t)hi;
          *reinterpret_cast<uint16_t*>(at + lo_off) = (uint16_t)lo;
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(smem_u32(&sm.p_full[sb]));
        if (j == pc.a) {      // while the tile's products run
          if (nu > 0 && !finish()) {
            ok = false;
            break;
          }
          more = walk.next(a, rows, nxt);
        }
      }
      if (!ok) break;
      fpc = pc;
      fhd = paged_head(a, pc.row, pc.sub, NQ);
      ffolded = folded;
      folded = false;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        if (row == 0) sm.base[nu & 1u][h] = m[h];
        fl[h] = l[h];
      }
      ++nu;
    }
    if (ok && nu > 0) finish();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// 4-D bf16 map: innermost D (boxes of 64, 128-byte swizzle), then three
// dimensions with strides in elements and box sizes.
static bool paged_map(CUtensorMap* m, const void* base, int D, const long long (&dim)[3], const long long (&stride)[3],
                      const int (&box)[3], CUtensorMapL2promotion promotion = CU_TENSOR_MAP_L2_PROMOTION_L2_256B) {
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)dim[0], (cuuint64_t)dim[1], (cuuint64_t)dim[2]};
  cuuint64_t strides[3];
  for (int i = 0; i < 3; ++i) strides[i] = (cuuint64_t)(dim[i] > 1 ? stride[i] : D) * 2;   // of one entry: any will do
  const cuuint32_t boxes[4] = {64, (cuuint32_t)box[0], (cuuint32_t)box[1], (cuuint32_t)box[2]};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, boxes, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, promotion,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int G, int DH>
static cudaError_t launch_paged_tc(const PagedDecodeArgs& a, cudaStream_t st) {
  CUtensorMap tq, tk, tv;
  PagedMaps maps;
  maps.head_outer = a.pool.head > a.pool.token;
  maps.q_rows = a.G < pdt::NQ ? a.G : pdt::NQ;
  const int ps = 1 << a.ps_log2, rows = ps < kPagedTile ? ps : kPagedTile;
  if (!paged_map(&tq, a.q, DH, {a.Hq, a.B, 1}, {a.q_h, a.q_b, a.q_b}, {maps.q_rows, 1, 1})) return cudaErrorInvalidValue;
  const PoolStrides& p = a.pool;
  // Heads of 64 beside each other: 128-byte rows, of which fetches of 256 bytes bring the neighbour's too
  // (56 sequences of 16,000 keys: 4 kv heads 393 us with 256, 268 with 128; 8 kv heads 419 and 326).
  const CUtensorMapL2promotion fetch = DH == 64 && p.token > DH ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                                : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  for (int i = 0; i < 2; ++i) {
    const void* base = i ? a.v : a.k;
    CUtensorMap* m = i ? &tv : &tk;
    if (!(maps.head_outer
              ? paged_map(m, base, DH, {ps, a.Hkv, a.num_pages}, {p.token, p.head, p.page}, {rows, 1, 1}, fetch)
              : paged_map(m, base, DH, {a.Hkv, ps, a.num_pages}, {p.head, p.token, p.page}, {1, rows, 1}, fetch)))
      return cudaErrorInvalidValue;
  }
  constexpr int smem = sizeof(PagedSmem<G, DH>) + 1024;
  static_assert(sizeof(PagedSmem<G, DH>) + 1024 <= 232448, "shared memory of a CTA");
  auto kern = paged_decode_kernel<G, DH>;
  const cudaError_t e = paged_raise_smem<smem>(kern);
  if (e != cudaSuccess) return e;
  const int grid = num_sms() < kPagedMaxCtas ? num_sms() : kPagedMaxCtas;
  return paged_launch(kern, grid, pdt::THREADS, smem, st, tq, tk, tv, a, maps);
}

cudaError_t launch_paged_decode(const PagedDecodeArgs& args, cudaStream_t st) {
  PagedDecodeArgs a = args;
  a.ngrp = (a.G + pdt::NQ - 1) / pdt::NQ;
  auto pick = [&](auto d) -> cudaError_t {
    constexpr int DD = decltype(d)::value;
    if (a.G == 1) return launch_paged_tc<1, DD>(a, st);
    if (a.G == 2) return launch_paged_tc<2, DD>(a, st);
    if (a.G <= 4) return launch_paged_tc<4, DD>(a, st);
    if (a.G <= 8) return launch_paged_tc<8, DD>(a, st);
    return launch_paged_tc<16, DD>(a, st);
  };
  return a.D == 64 ? pick(std::integral_constant<int, 64>{}) : pick(std::integral_constant<int, 128>{});
}

}  // namespace ra
