// C ABI of the paged-cache operators (declared in include/ring_attn.h):
// argument checks and dispatch.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/ring_attn.h"
#include "kernels.h"
#include "paged.h"

using namespace ra;

namespace {

bool aligned(const void* p, unsigned a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

ring_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return RING_OK;
  if (e == cudaErrorNotSupported) return RING_EUNSUPPORTED;
  if (e == cudaErrorInvalidValue) return RING_EINVAL;
  return RING_ECUDA;
}

// log2 of a page size: a power of two in [RING_PAGE_MIN, RING_PAGE_MAX]; -1 otherwise.
int page_log2(int ps) {
  if (ps < RING_PAGE_MIN || ps > RING_PAGE_MAX || (ps & (ps - 1))) return -1;
  int l = 0;
  while ((1 << l) < ps) ++l;
  return l;
}

bool good_dtype(int dtype) { return dtype == RING_BF16 || dtype == RING_FP32; }
int elem_bytes(int dtype) { return dtype == RING_BF16 ? 2 : 4; }

// A sequence's positions, and the slots of a pool, are 32-bit numbers.
bool table_fits(int W, int ps_log2) { return ((long long)W << ps_log2) <= 0x7fffff00LL; }

// Strides (elements) of rows of 16-byte pieces, far below 2^40 bytes.
bool good_stride(size_t s, int eb) { return s < (size_t(1) << 36) && (s * eb) % 16 == 0; }

// Strides of [n, heads, D] rows.
bool good_rows(size_t sn, size_t sh, int n, int heads, int D, int eb) {
  return good_stride(sn, eb) && good_stride(sh, eb) && (n == 1 || sn >= (size_t)D) && (heads == 1 || sh >= (size_t)D);
}

ring_status pool_check(const void* pool, int num_pages, int ps_log2, int Hkv, int D, size_t sp, size_t st, size_t sh,
                       int dtype, PoolStrides* out) {
  if (!aligned(pool, 16) || num_pages < 1 || Hkv < 1 || D < 1 || !good_dtype(dtype)) return RING_EINVAL;
  if (!table_fits(num_pages, ps_log2)) return RING_EINVAL;
  if (D != 64 && D != 128) return RING_EUNSUPPORTED;
  const int eb = elem_bytes(dtype);
  if (!good_stride(sp, eb) || !good_stride(st, eb) || !good_stride(sh, eb)) return RING_EINVAL;
  // rows next to each other in any dimension do not overlap (strides of two dimensions together are not compared)
  if (st < (size_t)D || (Hkv > 1 && sh < (size_t)D) || (num_pages > 1 && sp < (size_t)D)) return RING_EINVAL;
  out->page = (long long)sp;
  out->token = (long long)st;
  out->head = (long long)sh;
  return RING_OK;
}

}  // namespace

extern "C" {

ring_status ring_attn_page_extend(int32_t* seq_lens, const int32_t* new_lens, int32_t* block_table,
                                  const int32_t* free_pages, int32_t* n_free, int32_t* slot_map, int32_t* start_lens,
                                  int32_t* cu_new, int B, int W, size_t table_stride, int page_size, int max_free,
                                  int max_tokens, void* stream) {
  if (!aligned(seq_lens, 4) || !aligned(new_lens, 4) || !aligned(block_table, 4) || !aligned(free_pages, 4) ||
      !aligned(n_free, 4) || !aligned(slot_map, 4) || !aligned(start_lens, 4) || !aligned(cu_new, 4))
    return RING_EINVAL;
  if (B < 1 || W < 1 || max_free < 1 || max_tokens < 1 || page_size < 1 || table_stride < (size_t)W) return RING_EINVAL;
  const int pl = page_log2(page_size);
  if (pl < 0) return RING_EUNSUPPORTED;
  if (B > kPagedMaxSeqs || !table_fits(W, pl) || table_stride >= (size_t(1) << 32)) return RING_EINVAL;
  ExtendArgs a{};
  a.seq_lens = seq_lens; a.new_lens = new_lens; a.table = block_table; a.free_pages = free_pages; a.n_free = n_free;
  a.slot_map = slot_map; a.start_lens = start_lens; a.cu_new = cu_new;
  a.table_stride = (long long)table_stride;
  a.B = B; a.W = W; a.ps_log2 = pl; a.max_free = max_free; a.max_tokens = max_tokens;
  a.err = capacity_word();
  return from_cuda(launch_page_extend(a, reinterpret_cast<cudaStream_t>(stream)));
}

ring_status ring_attn_page_trim(int32_t* seq_lens, const int32_t* keep_lens, const int32_t* block_table,
                                int32_t* free_pages, int32_t* n_free, int B, int W, size_t table_stride,
                                int page_size, int max_free, void* stream) {
  if (!aligned(seq_lens, 4) || !aligned(keep_lens, 4) || !aligned(block_table, 4) || !aligned(free_pages, 4) ||
      !aligned(n_free, 4))
    return RING_EINVAL;
  if (B < 1 || W < 1 || max_free < 1 || page_size < 1 || table_stride < (size_t)W) return RING_EINVAL;
  const int pl = page_log2(page_size);
  if (pl < 0) return RING_EUNSUPPORTED;
  if (B > kPagedMaxSeqs || !table_fits(W, pl) || table_stride >= (size_t(1) << 32)) return RING_EINVAL;
  TrimArgs a{};
  a.seq_lens = seq_lens; a.keep_lens = keep_lens; a.table = block_table; a.free_pages = free_pages; a.n_free = n_free;
  a.table_stride = (long long)table_stride;
  a.B = B; a.W = W; a.ps_log2 = pl; a.max_free = max_free;
  a.err = capacity_word();
  return from_cuda(launch_page_trim(a, reinterpret_cast<cudaStream_t>(stream)));
}

ring_status ring_attn_paged_append(void* k_pool, void* v_pool, const void* k_new, const void* v_new,
                                   const int32_t* slot_map, int T, int Hkv, int D, int num_pages, int page_size,
                                   size_t stride_page, size_t stride_token, size_t stride_head, size_t new_token,
                                   size_t new_head, int dtype, void* stream) {
  if (!aligned(v_pool, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(slot_map, 4)) return RING_EINVAL;
  if (T < 1 || page_size < 1) return RING_EINVAL;
  const int pl = page_log2(page_size);
  if (pl < 0) return RING_EUNSUPPORTED;
  PagedAppendArgs a{};
  const ring_status rs = pool_check(k_pool, num_pages, pl, Hkv, D, stride_page, stride_token, stride_head, dtype,
                                    &a.pool);
  if (rs != RING_OK) return rs;
  a.elem_bytes = elem_bytes(dtype);
  if (!good_rows(new_token, new_head, T, Hkv, D, a.elem_bytes)) return RING_EINVAL;
  if ((long long)Hkv * D > (1LL << 24)) return RING_EINVAL;
  a.k_pool = k_pool; a.v_pool = v_pool; a.k_new = k_new; a.v_new = v_new; a.slot_map = slot_map;
  a.new_token = (long long)new_token;
  a.new_head = (long long)new_head;
  a.T = T; a.Hkv = Hkv; a.D = D; a.num_pages = num_pages; a.ps_log2 = pl;
  return from_cuda(launch_paged_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t ring_attn_decode_paged_workspace_bytes(int D) {
  if (D != 64 && D != 128) return 0;
  return paged_decode_workspace_bytes(D);
}

ring_status ring_attn_decode_paged(const void* q, const void* k_pool, const void* v_pool, const int32_t* block_table,
                                   const int32_t* seq_lens, const int32_t* sel, const int32_t* n_sel, void* out,
                                   float* out_lse, int B, int Hq, int Hkv, int D, int num_pages, int page_size, int W,
                                   int K, size_t q_stride_b, size_t q_stride_h, size_t stride_page,
                                   size_t stride_token, size_t stride_head, size_t table_stride, float scale,
                                   int dtype, int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!aligned(q, 16) || !aligned(v_pool, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(out, 16))
    return RING_EINVAL;
  if (out_lse && !aligned(out_lse, 4)) return RING_EINVAL;
  if ((sel == nullptr) != (n_sel == nullptr)) return RING_EINVAL;
  if (sel && (!aligned(sel, 4) || !aligned(n_sel, 4) || K < 1)) return RING_EINVAL;
  if (B < 1 || Hq < 1 || Hkv < 1 || W < 1 || page_size < 1 || Hq % Hkv || table_stride < (size_t)W) return RING_EINVAL;
  if (!(scale > 0.f) || !std::isfinite(scale)) return RING_EINVAL;
  if (!good_dtype(out_dtype)) return RING_EINVAL;
  const int pl = page_log2(page_size);
  if (pl < 0) return RING_EUNSUPPORTED;
  PagedDecodeArgs a{};
  const ring_status rs = pool_check(k_pool, num_pages, pl, Hkv, D, stride_page, stride_token, stride_head, dtype,
                                    &a.pool);
  if (rs != RING_OK) return rs;
  if (dtype == RING_FP32 && out_dtype != RING_FP32) return RING_EUNSUPPORTED;
  const int eb = elem_bytes(dtype);
  if (!good_rows(q_stride_b, q_stride_h, B, Hq, D, eb)) return RING_EINVAL;
  if (!table_fits(W, pl) || table_stride >= (size_t(1) << 32) || (sel && !table_fits(K, pl))) return RING_EINVAL;
  // outputs, and the call's units (per segment its tiles and its fixed cost), count in 32 bits
  if ((long long)B * Hq > 0x7fffffffLL / D) return RING_EINVAL;
  const long long keys = (long long)(sel ? K : W) << pl;
  const int G = Hq / Hkv, group = dtype == RING_BF16 ? kPagedHeads : kPagedSimtHeads;
  const int seg_cost = dtype == RING_BF16 ? paged_seg_cost(G) : kPagedSimtSegCost;
  const long long segs = (long long)B * Hkv * ((G + group - 1) / group);
  if (segs * ((keys + kPagedTile - 1) / kPagedTile + seg_cost) > 0x7fffffffLL) return RING_EINVAL;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < paged_decode_workspace_bytes(D))
    return RING_EINVAL;
  a.q = q; a.k = k_pool; a.v = v_pool; a.table = block_table; a.seq_lens = seq_lens; a.sel = sel; a.n_sel = n_sel;
  a.out = out; a.out_lse = out_lse;
  paged_decode_workspace_split(workspace, &a.ws_part, &a.ws_count);
  a.q_b = (long long)q_stride_b;
  a.q_h = (long long)q_stride_h;
  a.table_stride = (long long)table_stride;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.num_pages = num_pages; a.ps_log2 = pl; a.W = W; a.K = sel ? K : 0;
  a.G = G;
  a.scale = scale;
  a.out_fp32 = out_dtype == RING_FP32;
  a.err = error_word();
  cudaStream_t strm = reinterpret_cast<cudaStream_t>(stream);
  return from_cuda(dtype == RING_BF16 ? launch_paged_decode(a, strm) : launch_paged_decode_simt(a, strm));
}

ring_status ring_attn_page_bounds(const void* k_pool, void* bounds, const int32_t* block_table,
                                  const int32_t* seq_lens, const int32_t* start_lens, int B, int Hkv, int D,
                                  int num_pages, int page_size, int W, size_t stride_page, size_t stride_token,
                                  size_t stride_head, size_t table_stride, int dtype, void* stream) {
  if (!aligned(bounds, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4)) return RING_EINVAL;
  if (start_lens && !aligned(start_lens, 4)) return RING_EINVAL;
  if (B < 1 || W < 1 || page_size < 1 || table_stride < (size_t)W) return RING_EINVAL;
  const int pl = page_log2(page_size);
  if (pl < 0 || B > 65535) return RING_EUNSUPPORTED;
  BoundsArgs a{};
  const ring_status rs = pool_check(k_pool, num_pages, pl, Hkv, D, stride_page, stride_token, stride_head, dtype,
                                    &a.pool);
  if (rs != RING_OK) return rs;
  if (!table_fits(W, pl) || table_stride >= (size_t(1) << 32)) return RING_EINVAL;
  if ((long long)Hkv * D > 0x7fffffffLL / elem_bytes(dtype)) return RING_EINVAL;    // bytes of a token's row
  a.k = k_pool; a.bounds = bounds; a.table = block_table; a.seq_lens = seq_lens; a.start_lens = start_lens;
  a.table_stride = (long long)table_stride;
  a.B = B; a.Hkv = Hkv; a.D = D; a.num_pages = num_pages; a.ps_log2 = pl; a.W = W; a.elem_bytes = elem_bytes(dtype);
  return from_cuda(launch_page_bounds(a, reinterpret_cast<cudaStream_t>(stream)));
}

ring_status ring_attn_page_scores(const void* q, const void* bounds, const int32_t* block_table,
                                  const int32_t* seq_lens, float* scores, int B, int Hq, int Hkv, int D, int num_pages,
                                  int page_size, int W, size_t q_stride_b, size_t q_stride_h, size_t table_stride,
                                  int dtype, void* stream) {
  if (!aligned(q, 16) || !aligned(bounds, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(scores, 4))
    return RING_EINVAL;
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || D < 1 || W < 1 || num_pages < 1 || page_size < 1 ||
      table_stride < (size_t)W || !good_dtype(dtype))
    return RING_EINVAL;
  const int pl = page_log2(page_size);
  if (pl < 0 || (D != 64 && D != 128) || (long long)B * Hkv > 65535) return RING_EUNSUPPORTED;
  if (Hq / Hkv > 64) return RING_EUNSUPPORTED;    // the group's queries sit in shared memory
  const int eb = elem_bytes(dtype);
  if (!good_rows(q_stride_b, q_stride_h, B, Hq, D, eb)) return RING_EINVAL;
  if (!table_fits(W, pl) || !table_fits(num_pages, pl) || table_stride >= (size_t(1) << 32)) return RING_EINVAL;
  ScoresArgs a{};
  a.q = q; a.bounds = bounds; a.table = block_table; a.seq_lens = seq_lens; a.scores = scores;
  a.q_b = (long long)q_stride_b;
  a.q_h = (long long)q_stride_h;
  a.table_stride = (long long)table_stride;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.num_pages = num_pages; a.ps_log2 = pl; a.W = W;
  return from_cuda(launch_page_scores(a, dtype == RING_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

ring_status ring_attn_page_select(const float* scores, const int32_t* seq_lens, int32_t* sel, int32_t* n_sel, int B,
                                  int Hkv, int W, int page_size, int K, int keep_first, int keep_last, void* stream) {
  if (!aligned(scores, 4) || !aligned(seq_lens, 4) || !aligned(sel, 4) || !aligned(n_sel, 4)) return RING_EINVAL;
  if (B < 1 || Hkv < 1 || W < 1 || K < 1 || page_size < 1 || keep_first < 0 || keep_last < 0 ||
      (long long)keep_first + keep_last > K)
    return RING_EINVAL;
  const int pl = page_log2(page_size);
  if (pl < 0) return RING_EUNSUPPORTED;
  if (!table_fits(W, pl) || !table_fits(K, pl) || (long long)B * Hkv > 0x7fffffffLL) return RING_EINVAL;
  SelectArgs a{scores, seq_lens, sel, n_sel, B, Hkv, W, pl, K, keep_first, keep_last};
  return from_cuda(launch_page_select(a, reinterpret_cast<cudaStream_t>(stream)));
}

ring_status ring_attn_paged_packed(int call, const int64_t* args, int n, void* stream) {
  if (!args || (reinterpret_cast<uintptr_t>(args) & 7u)) return RING_EINVAL;
  // per call, in order: how many words, and which of them are ints (bit i: word i), which may not be cut
  static constexpr struct {
    int n;
    uint32_t ints;
  } kWords[] = {{14, 0x3b00u}, {10, 0x360u}, {16, 0x83e0u}, {28, 0x301fe00u}, {16, 0x87e0u}, {16, 0x8fe0u}, {11, 0x7f0u}};
  if (call < 0 || call > RING_PAGE_SELECT || n != kWords[call].n) return RING_EINVAL;
  for (int i = 0; i < n; ++i)
    if ((kWords[call].ints >> i & 1u) && args[i] != static_cast<int>(args[i])) return RING_EINVAL;
  // the arguments in order: pointers, ints and sizes as they are, the scale as the bits of a double
  auto ptr = [&](int i) { return reinterpret_cast<void*>(static_cast<intptr_t>(args[i])); };
  auto i32 = [&](int i) { return reinterpret_cast<int32_t*>(ptr(i)); };
  auto f32 = [&](int i) { return reinterpret_cast<float*>(ptr(i)); };
  auto num = [&](int i) { return static_cast<int>(args[i]); };
  auto size = [&](int i) { return static_cast<size_t>(args[i]); };
  switch (call) {
    case RING_PAGE_EXTEND:
      return ring_attn_page_extend(i32(0), i32(1), i32(2), i32(3), i32(4), i32(5), i32(6), i32(7), num(8), num(9),
                                   size(10), num(11), num(12), num(13), stream);
    case RING_PAGE_TRIM:
      return ring_attn_page_trim(i32(0), i32(1), i32(2), i32(3), i32(4), num(5), num(6), size(7), num(8), num(9),
                                 stream);
    case RING_PAGED_APPEND:
      return ring_attn_paged_append(ptr(0), ptr(1), ptr(2), ptr(3), i32(4), num(5), num(6), num(7), num(8), num(9),
                                    size(10), size(11), size(12), size(13), size(14), num(15), stream);
    case RING_DECODE_PAGED: {
      double scale;
      memcpy(&scale, args + 23, sizeof(scale));
      return ring_attn_decode_paged(ptr(0), ptr(1), ptr(2), i32(3), i32(4), i32(5), i32(6), ptr(7), f32(8), num(9),
                                    num(10), num(11), num(12), num(13), num(14), num(15), num(16), size(17), size(18),
                                    size(19), size(20), size(21), size(22), static_cast<float>(scale), num(24), num(25),
                                    ptr(26), size(27), stream);
    }
    case RING_PAGE_BOUNDS:
      return ring_attn_page_bounds(ptr(0), ptr(1), i32(2), i32(3), i32(4), num(5), num(6), num(7), num(8), num(9),
                                   num(10), size(11), size(12), size(13), size(14), num(15), stream);
    case RING_PAGE_SCORES:
      return ring_attn_page_scores(ptr(0), ptr(1), i32(2), i32(3), f32(4), num(5), num(6), num(7), num(8), num(9),
                                   num(10), num(11), size(12), size(13), size(14), num(15), stream);
    case RING_PAGE_SELECT:
      return ring_attn_page_select(f32(0), i32(1), i32(2), i32(3), num(4), num(5), num(6), num(7), num(8), num(9),
                                   num(10), stream);
  }
  return RING_EINVAL;
}

}  // extern "C"
