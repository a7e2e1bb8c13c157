// Host-side launchers of the paged-cache operators (internal; the public ABI
// is include/ring_attn.h).
//
// A cache page holds `ps` tokens (a power of two); the pools k, v are
// [num_pages, ps, Hkv, D] with unit stride along D and the strides below
// (elements).  block_table[b][i] is the pool page of tokens
// [i*ps, (i+1)*ps) of sequence b.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

namespace ra {

// Launches with programmatic stream serialization: the kernel may start while
// the one before it on the stream finishes.  Every kernel launched so begins
// with paged_begin(), before it touches global memory.
template <typename... P, typename... A>
inline cudaError_t paged_launch(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

// Raises a kernel's shared-memory limit to kBytes, once per device.
template <int kBytes, typename Kern>
inline cudaError_t paged_raise_smem(Kern kern) {
  static std::atomic<const void*> raised[64];    // of every instantiation's type; a kernel is told by its address
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const void* k = reinterpret_cast<const void*>(kern);
  if (dev < 64 && raised[dev].load(std::memory_order_relaxed) == k) return cudaSuccess;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e == cudaSuccess && dev < 64) raised[dev].store(k, std::memory_order_relaxed);
  return e;
}

struct PoolStrides {
  long long page, token, head;   // elements
};

// ---- block tables and slot maps ----
constexpr int kPagedMaxSeqs = 0x7fffffff - 1024;   // sequences are counted in 32 bits, past the last of them by a block
struct ExtendArgs {
  int32_t* seq_lens;          // [B], advanced
  const int32_t* new_lens;    // [B]
  int32_t* table;             // [B, W], row stride table_stride
  const int32_t* free_pages;  // [max_free], a stack of n_free[0] pages
  int32_t* n_free;            // [1]
  int32_t* slot_map;          // [max_tokens]
  int32_t* start_lens;        // [B]
  int32_t* cu_new;            // [B + 1]
  long long table_stride;
  int B, W, ps_log2, max_free, max_tokens;
  unsigned int* err;          // capacity word
};
cudaError_t launch_page_extend(const ExtendArgs& a, cudaStream_t st);

struct TrimArgs {
  int32_t* seq_lens;         // [B], shortened
  const int32_t* keep_lens;  // [B]
  const int32_t* table;
  int32_t* free_pages;
  int32_t* n_free;
  long long table_stride;
  int B, W, ps_log2, max_free;
  unsigned int* err;          // capacity word
};
cudaError_t launch_page_trim(const TrimArgs& a, cudaStream_t st);

// ---- paged append ----
struct PagedAppendArgs {
  void* k_pool;
  void* v_pool;
  const void* k_new;          // [T, Hkv, D], strides below
  const void* v_new;
  const int32_t* slot_map;    // [T]; outside [0, num_pages*ps): not written
  PoolStrides pool;
  long long new_token, new_head;   // elements
  int T, Hkv, D, num_pages, ps_log2, elem_bytes;
};
cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t st);

// ---- paged decode ----
// The most CTAs a decode launch uses (one per SM of a B200); fixes the size of
// the workspace.
constexpr int kPagedMaxCtas = 148;
constexpr int kPagedTile = 128;       // keys per tile, the unit the work is split in
constexpr int kPagedHeads = 16;       // query heads a CTA works on at once (a head group)
constexpr int kPagedSimtHeads = 8;    // the same of the float32 kernel
// What a segment costs besides its tiles, in tiles, of G query heads per kv head (measured: see the kernels).
__host__ __device__ constexpr int paged_seg_cost(int G) { return G > 8 ? 2 : 1; }
constexpr int kPagedSimtSegCost = 2;

struct PagedDecodeArgs {
  const void* q;                // [B, Hq, D], strides q_b, q_h
  const void* k;
  const void* v;
  const int32_t* table;         // [B, W]
  const int32_t* seq_lens;      // [B]
  const int32_t* sel;           // null, or [B, Hkv, K]: the logical pages to read, entries outside the sequence ignored
  const int32_t* n_sel;         // [B, Hkv]
  void* out;                    // [B, Hq, D]
  float* out_lse;               // [B, Hq] or null
  float* ws_part;               // [2 kPagedMaxCtas][kPagedHeads][D] results of pieces, then their lse
  unsigned int* ws_count;       // [kPagedMaxCtas], zero between calls
  PoolStrides pool;
  long long q_b, q_h, table_stride;
  int B, Hq, Hkv, D, num_pages, ps_log2, W, K;
  int G;                        // query heads per kv head
  int ngrp;                     // head groups per kv head
  float scale;
  int out_fp32;
  unsigned int* err;
};
size_t paged_decode_workspace_bytes(int D);
void paged_decode_workspace_split(void* ws, float** part, unsigned int** count);
cudaError_t launch_paged_decode(const PagedDecodeArgs& a, cudaStream_t st);        // bf16, tensor cores
cudaError_t launch_paged_decode_simt(const PagedDecodeArgs& a, cudaStream_t st);   // float32, CUDA cores

// ---- page bounds, scores, selection ----
struct BoundsArgs {
  const void* k;
  void* bounds;                 // [num_pages, Hkv, 2, D]: minimum, maximum
  const int32_t* table;
  const int32_t* seq_lens;
  const int32_t* start_lens;    // [B] or null
  PoolStrides pool;
  long long table_stride;
  int B, Hkv, D, num_pages, ps_log2, W, elem_bytes;
};
cudaError_t launch_page_bounds(const BoundsArgs& a, cudaStream_t st);

struct ScoresArgs {
  const void* q;
  const void* bounds;
  const int32_t* table;
  const int32_t* seq_lens;
  float* scores;                // [B, Hkv, W]
  long long q_b, q_h, table_stride;
  int B, Hq, Hkv, D, num_pages, ps_log2, W;
};
cudaError_t launch_page_scores(const ScoresArgs& a, bool bf16, cudaStream_t st);

struct SelectArgs {
  const float* scores;          // [B, Hkv, W]
  const int32_t* seq_lens;
  int32_t* sel;                 // [B, Hkv, K]
  int32_t* n_sel;               // [B, Hkv]
  int B, Hkv, W, ps_log2, K, keep_first, keep_last;
};
cudaError_t launch_page_select(const SelectArgs& a, cudaStream_t st);

}  // namespace ra
