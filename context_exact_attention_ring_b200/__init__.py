"""Exact ring attention on one B200 (sm_100a), emulating P virtual ranks.

A thin ctypes binding over ``libringattn_sm100a.so`` (C ABI in
``include/ring_attn.h``).  It only marshals arguments: torch tensors are
passed by device pointer and the current torch CUDA stream; every step of the
computation runs in the library's CUDA kernels.  There is no CPU fallback --
importing works without a GPU (for the host-side helpers), but every compute
call raises if the library or a CUDA device is missing.

Names follow the C ABI:
  ring_attn_fwd, ring_attn_fwd_counted, ring_attn_fwd_simt,
  ring_attn_state_init, ring_attn_step, ring_attn_state_finalize,
  ring_attn_decode_partial, ring_attn_merge, ring_attn_decode,
  ring_attn_decode_workspace_bytes, ring_attn_decode_fused,
  ring_attn_kv_append, ring_attn_sched_stats, ring_attn_device_error;
  ring_attn_page_extend, ring_attn_page_trim, ring_attn_paged_append,
  ring_attn_decode_paged, ring_attn_page_bounds, ring_attn_page_scores,
  ring_attn_page_select, ring_attn_paged_packed (the paged KV cache);
and ring_attention (RingAttnFunction), the forward and backward under autograd.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libringattn_sm100a.so")

RING_OK, RING_EINVAL, RING_EUNSUPPORTED, RING_ECUDA, RING_ETIMEOUT, RING_ECAPACITY = 0, -1, -2, -3, -4, -5
RING_CONTIGUOUS, RING_ZIGZAG, RING_STRIPED = 0, 1, 2
RING_MAX_CHUNKS_PER_RANK = 8
RING_BF16, RING_FP32 = 0, 1
LAYOUTS = {"contiguous": RING_CONTIGUOUS, "zigzag": RING_ZIGZAG, "striped": RING_STRIPED}


def ring_split(split: str, k: int = 0) -> int:
    """The C ABI's split code RING_SPLIT(split, k): k chunks per rank (0 = the split's default)."""
    return LAYOUTS[split] | (int(k) << 8)

EXPORTED = (
    "ring_attn_fwd", "ring_attn_fwd_counted", "ring_attn_fwd_simt", "ring_attn_state_init", "ring_attn_step",
    "ring_attn_state_finalize", "ring_attn_decode_partial", "ring_attn_decode_workspace_bytes", "ring_attn_decode",
    "ring_attn_merge", "ring_attn_sched_stats", "ring_attn_device_error", "ring_attn_strerror",
    "ring_attn_version", "ring_attn_built_arch", "ring_attn_selftest_wait", "ring_attn_decode_partial_noalloc",
    "ring_attn_decode_fused", "ring_attn_kv_append", "ring_attn_bwd", "ring_attn_bwd_delta",
    "ring_attn_bwd_workspace_bytes", "ring_attn_step_bwd", "ring_attn_bwd_simt",
    "ring_attn_page_extend", "ring_attn_page_trim", "ring_attn_paged_append", "ring_attn_decode_paged_workspace_bytes",
    "ring_attn_decode_paged", "ring_attn_page_bounds", "ring_attn_page_scores", "ring_attn_page_select",
    "ring_attn_paged_packed",
)


class RingError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {strerror(status)} ({status})")


class ChunkIds(ctypes.Structure):
    _fields_ = [("n_q", ctypes.c_int32), ("q", ctypes.c_int32 * RING_MAX_CHUNKS_PER_RANK),
                ("n_kv", ctypes.c_int32), ("kv", ctypes.c_int32 * RING_MAX_CHUNKS_PER_RANK),
                ("chunk_len", ctypes.c_int32), ("causal", ctypes.c_int32), ("stripes", ctypes.c_int32)]


_lib = None


def lib():
    """The loaded shared library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m context_exact_attention_ring_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    prefill = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, f32, i32]
    sig = {
        "ring_attn_fwd": prefill + [vp],
        "ring_attn_fwd_counted": prefill + [vp, vp],
        "ring_attn_fwd_simt": prefill + [vp],
        "ring_attn_state_init": [vp, vp, vp, i32, i32, i32, i32, vp],
        "ring_attn_step": [vp, vp, vp, vp, vp, vp, ctypes.POINTER(ChunkIds), i32, i32, i32, i32, f32, i32, vp],
        "ring_attn_state_finalize": [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp],
        "ring_attn_decode_partial": [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, i32, vp, sz, vp],
        "ring_attn_decode": [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, i32, vp, sz, vp],
        "ring_attn_decode_partial_noalloc": [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, i32, vp],
        "ring_attn_decode_fused": [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, i32, vp, sz,
                                   vp],
        "ring_attn_kv_append": [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, vp],
        "ring_attn_bwd": [vp] * 9 + [i32] * 8 + [f32, i32, vp, sz, vp],
        "ring_attn_bwd_simt": [vp] * 9 + [i32] * 8 + [f32, i32, vp, sz, vp],
        "ring_attn_bwd_delta": [vp, vp, vp, i32, i32, i32, i32, i32, vp],
        "ring_attn_step_bwd": [vp] * 9 + [ctypes.POINTER(ChunkIds), i32, i32, i32, i32, f32, i32, vp],
        "ring_attn_merge": [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp],
        "ring_attn_sched_stats": [i32, i32, i32, i32, i32, i32, vp, vp, vp, vp],
        "ring_attn_device_error": [ctypes.POINTER(ctypes.c_int)],
        "ring_attn_strerror": [i32],
        "ring_attn_version": [],
        "ring_attn_selftest_wait": [i32, vp],
        "ring_attn_built_arch": [],
        "ring_attn_page_extend": [vp] * 8 + [i32, i32, sz, i32, i32, i32, vp],
        "ring_attn_page_trim": [vp] * 5 + [i32, i32, sz, i32, i32, vp],
        "ring_attn_paged_append": [vp] * 5 + [i32] * 5 + [sz] * 5 + [i32, vp],
        "ring_attn_decode_paged": [vp] * 9 + [i32] * 8 + [sz] * 6 + [f32, i32, i32, vp, sz, vp],
        "ring_attn_page_bounds": [vp] * 5 + [i32] * 6 + [sz] * 4 + [i32, vp],
        "ring_attn_page_scores": [vp] * 5 + [i32] * 7 + [sz] * 3 + [i32, vp],
        "ring_attn_page_select": [vp] * 4 + [i32] * 7 + [vp],
        "ring_attn_paged_packed": [i32, vp, i32, vp],
    }
    for name, args in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    L.ring_attn_strerror.restype = ctypes.c_char_p
    L.ring_attn_decode_workspace_bytes.argtypes = [i32] * 6
    L.ring_attn_decode_workspace_bytes.restype = sz
    L.ring_attn_bwd_workspace_bytes.argtypes = [i32] * 3
    L.ring_attn_bwd_workspace_bytes.restype = sz
    L.ring_attn_decode_paged_workspace_bytes.argtypes = [i32]
    L.ring_attn_decode_paged_workspace_bytes.restype = sz
    _lib = L
    return L


def strerror(status: int) -> str:
    try:
        return lib().ring_attn_strerror(int(status)).decode()
    except RuntimeError:
        return str(status)


def _check(status: int, what: str):
    if status != RING_OK:
        raise RingError(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _cuda(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must live on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return RING_BF16
    if t.dtype == torch.float32:
        return RING_FP32
    raise ValueError(f"unsupported dtype {t.dtype}")


def _layout(layout) -> int:
    """A split code from 'contiguous' | 'zigzag' | 'striped', optionally with the
    chunks per rank appended ('zigzag4', 'contiguous2'), or an int code."""
    if not isinstance(layout, str):
        return int(layout)
    name = layout.rstrip("0123456789")
    k = layout[len(name):]
    if name not in LAYOUTS:
        raise ValueError(f"unknown split {layout!r}")
    return ring_split(name, int(k) if k else 0)


def _prefill(name, q, k, v, P, causal, layout, scale, out, lse, extra=()):
    _cuda(q, k, v, out, lse)
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    if k.shape != (B, S, Hkv, D) or v.shape != k.shape or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q [B,S,Hq,D], k/v [B,S,Hkv,D] of one dtype expected")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, S), device=q.device, dtype=torch.float32)
    st = getattr(lib(), name)(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, S, D, int(P),
                               int(bool(causal)), _layout(layout), scale, _dtype_code(q), *extra, _stream())
    _check(st, name)
    return out, lse


def ring_attn_fwd(q, k, v, P, causal=True, layout="zigzag", scale=None, out=None, lse=None):
    """Whole ring (all P virtual ranks) in one launch.  Returns (out, lse)."""
    return _prefill("ring_attn_fwd", q, k, v, P, causal, layout, scale, out, lse)


def ring_attn_fwd_counted(q, k, v, P, causal=True, layout="zigzag", scale=None, out=None, lse=None, counters=None):
    """ring_attn_fwd plus the device-side work counters [full, partial, pairs of rank 0..P-1]."""
    if counters is None:
        counters = torch.zeros(2 + int(P), device=q.device, dtype=torch.int64)
    out, lse = _prefill("ring_attn_fwd_counted", q, k, v, P, causal, layout, scale, out, lse,
                        extra=(_ptr(counters),))
    return out, lse, counters


def ring_attn_fwd_simt(q, k, v, P, causal=True, layout="zigzag", scale=None, out=None, lse=None):
    """The CUDA-core cross-check path of ring_attn_fwd."""
    return _prefill("ring_attn_fwd_simt", q, k, v, P, causal, layout, scale, out, lse)


def ring_attn_bwd_delta(out, dout, delta=None):
    """delta [B,Hq,S] = rowsum(dout * out) for out, dout [B,S,Hq,D]."""
    _cuda(out, dout, delta)
    B, S, Hq, D = out.shape
    if delta is None:
        delta = torch.empty((B, Hq, S), device=out.device, dtype=torch.float32)
    _check(lib().ring_attn_bwd_delta(_ptr(out), _ptr(dout), _ptr(delta), B, Hq, S, D, _dtype_code(out), _stream()),
           "ring_attn_bwd_delta")
    return delta


def ring_attn_bwd(q, k, v, out, lse, dout, P, causal=True, layout="zigzag", scale=None, dq=None, dk=None, dv=None,
                  workspace=None, _name="ring_attn_bwd"):
    """Gradients (dq, dk, dv) of the whole ring for the output gradient dout."""
    _cuda(q, k, v, out, lse, dout, dq, dk, dv, workspace)
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    if out.shape != q.shape or dout.shape != q.shape or dout.dtype != q.dtype or out.dtype != q.dtype:
        raise ValueError("out and dout must match q")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        workspace = torch.empty(int(lib().ring_attn_bwd_workspace_bytes(B, Hq, S)), device=q.device,
                                dtype=torch.uint8)
    st = getattr(lib(), _name)(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                               _ptr(dv), B, Hq, Hkv, S, D, int(P), int(bool(causal)), _layout(layout), scale,
                               _dtype_code(q), _ptr(workspace), workspace.numel(), _stream())
    _check(st, _name)
    return dq, dk, dv


def ring_attn_bwd_simt(q, k, v, out, lse, dout, P, causal=True, layout="zigzag", scale=None, dq=None, dk=None,
                       dv=None, workspace=None):
    """The CUDA-core cross-check path of ring_attn_bwd."""
    return ring_attn_bwd(q, k, v, out, lse, dout, P, causal, layout, scale, dq, dk, dv, workspace,
                         _name="ring_attn_bwd_simt")


def ring_attn_step_bwd(q_shard, kchunk, vchunk, dout_shard, lse, delta, dq_acc, dk_acc, dv_acc, q_ids, kv_ids,
                       chunk_len, causal=True, scale=None, stripes=0):
    """One backward hop: add this block's share to dq_acc and the shard's share
    to dk_acc, dv_acc (float32, in place)."""
    _cuda(q_shard, kchunk, vchunk, dout_shard, lse, delta, dq_acc, dk_acc, dv_acc)
    B, Sq, Hq, D = q_shard.shape
    Hkv = kchunk.shape[2]
    ids = _chunk_ids(q_ids, kv_ids, chunk_len, causal, stripes)
    if Sq != len(q_ids) * chunk_len or kchunk.shape[1] != len(kv_ids) * chunk_len:
        raise ValueError("shard / chunk buffers do not match the chunk ids")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    st = lib().ring_attn_step_bwd(_ptr(q_shard), _ptr(kchunk), _ptr(vchunk), _ptr(dout_shard), _ptr(lse),
                                  _ptr(delta), _ptr(dq_acc), _ptr(dk_acc), _ptr(dv_acc), ctypes.byref(ids), B, Hq,
                                  Hkv, D, scale, _dtype_code(q_shard), _stream())
    _check(st, "ring_attn_step_bwd")


def _chunk_ids(q_ids, kv_ids, chunk_len, causal, stripes):
    if not (1 <= len(q_ids) <= RING_MAX_CHUNKS_PER_RANK and 1 <= len(kv_ids) <= RING_MAX_CHUNKS_PER_RANK):
        raise ValueError(f"1..{RING_MAX_CHUNKS_PER_RANK} chunk ids expected")
    ids = ChunkIds()
    ids.n_q = len(q_ids)
    ids.n_kv = len(kv_ids)
    for i, c in enumerate(q_ids):
        ids.q[i] = int(c)
    for i, c in enumerate(kv_ids):
        ids.kv[i] = int(c)
    ids.chunk_len = int(chunk_len)
    ids.causal = int(bool(causal))
    ids.stripes = int(stripes)
    return ids


def ring_attn_state_init(m, l, O):
    _cuda(m, l, O)
    B, Hq, S = m.shape
    _check(lib().ring_attn_state_init(_ptr(m), _ptr(l), _ptr(O), B, Hq, S, O.shape[-1], _stream()),
           "ring_attn_state_init")


def new_state(B, Hq, S_loc, D, device="cuda"):
    """Allocate (with torch) and initialise a ring state (m, l, O)."""
    m = torch.empty((B, Hq, S_loc), device=device, dtype=torch.float32)
    l = torch.empty_like(m)
    O = torch.empty((B, S_loc, Hq, D), device=device, dtype=torch.float32)
    ring_attn_state_init(m, l, O)
    return m, l, O


def ring_attn_step(q_shard, kchunk, vchunk, m, l, O, q_ids, kv_ids, chunk_len, causal=True, scale=None, stripes=0):
    """One ring hop: fold the held K/V chunks (global ids kv_ids) into the
    state of the query shard (global chunk ids q_ids), in place.  With
    stripes=P the shard and the block are stripes of the striped split and
    q_ids / kv_ids hold the two ranks."""
    _cuda(q_shard, kchunk, vchunk, m, l, O)
    B, Sq, Hq, D = q_shard.shape
    Hkv = kchunk.shape[2]
    ids = _chunk_ids(q_ids, kv_ids, chunk_len, causal, stripes)
    if Sq != len(q_ids) * chunk_len or kchunk.shape[1] != len(kv_ids) * chunk_len:
        raise ValueError("shard / chunk buffers do not match the chunk ids")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    st = lib().ring_attn_step(_ptr(q_shard), _ptr(kchunk), _ptr(vchunk), _ptr(m), _ptr(l), _ptr(O),
                              ctypes.byref(ids), B, Hq, Hkv, D, scale, _dtype_code(q_shard), _stream())
    _check(st, "ring_attn_step")


def ring_attn_state_finalize(m, l, O, dtype=torch.bfloat16, out=None, lse=None):
    _cuda(m, l, O)
    B, S, Hq, D = O.shape
    if out is None:
        out = torch.empty((B, S, Hq, D), device=O.device, dtype=dtype)
    if lse is None:
        lse = torch.empty((B, Hq, S), device=O.device, dtype=torch.float32)
    st = lib().ring_attn_state_finalize(_ptr(m), _ptr(l), _ptr(O), _ptr(out), _ptr(lse), B, Hq, S, D,
                                        _dtype_code(out), _stream())
    _check(st, "ring_attn_state_finalize")
    return out, lse


def ring_attn_decode_workspace_bytes(B, Hq, Hkv, Smax, D, P) -> int:
    return int(lib().ring_attn_decode_workspace_bytes(B, Hq, Hkv, Smax, D, P))


def decode_workspace(B, Hq, Hkv, Smax, D, P, device="cuda"):
    """A zeroed workspace for the decode calls (allocated with torch)."""
    n = ring_attn_decode_workspace_bytes(B, Hq, Hkv, Smax, D, P)
    if n == 0:
        raise ValueError("bad decode sizes")
    return torch.zeros(n, device=device, dtype=torch.uint8)


def _decode_shapes(q, k, seqlens, P):
    B, Hq, D = q.shape
    _, Smax, Hkv, _ = k.shape
    if seqlens.dtype != torch.int32 or seqlens.shape != (B,):
        raise ValueError("seqlens must be int32 [B]")
    return B, Hq, Hkv, Smax, D


def ring_attn_decode_partial(q, k, v, seqlens, P, scale=None, partials=None, part_lse=None, workspace=None):
    _cuda(q, k, v, seqlens, partials, part_lse, workspace)
    B, Hq, Hkv, Smax, D = _decode_shapes(q, k, seqlens, P)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if partials is None:
        partials = torch.empty((B, Hq, P, D), device=q.device, dtype=torch.float32)
    if part_lse is None:
        part_lse = torch.empty((B, Hq, P), device=q.device, dtype=torch.float32)
    if workspace is None:
        workspace = decode_workspace(B, Hq, Hkv, Smax, D, P, q.device)
    st = lib().ring_attn_decode_partial(_ptr(q), _ptr(k), _ptr(v), _ptr(seqlens), _ptr(partials), _ptr(part_lse),
                                        B, Hq, Hkv, Smax, D, int(P), scale, _dtype_code(q), _ptr(workspace),
                                        workspace.numel(), _stream())
    _check(st, "ring_attn_decode_partial")
    return partials, part_lse


def ring_attn_decode_partial_noalloc(q, k, v, seqlens, P, scale=None, partials=None, part_lse=None):
    """ring_attn_decode_partial using the library's fixed scratch array (no
    workspace, no allocation inside the call; see include/ring_attn.h).
    Pass preallocated `partials` and `part_lse` to avoid torch allocations."""
    _cuda(q, k, v, seqlens, partials, part_lse)
    B, Hq, Hkv, Smax, D = _decode_shapes(q, k, seqlens, P)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if partials is None:
        partials = torch.empty((B, Hq, P, D), device=q.device, dtype=torch.float32)
    if part_lse is None:
        part_lse = torch.empty((B, Hq, P), device=q.device, dtype=torch.float32)
    st = lib().ring_attn_decode_partial_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(seqlens), _ptr(partials),
                                                _ptr(part_lse), B, Hq, Hkv, Smax, D, int(P), scale, _dtype_code(q),
                                                _stream())
    _check(st, "ring_attn_decode_partial_noalloc")
    return partials, part_lse


def ring_attn_merge(partials, part_lse, out=None, out_lse=None, dtype=torch.bfloat16):
    _cuda(partials, part_lse, out, out_lse)
    B, Hq, P, D = partials.shape
    if out is None:
        out = torch.empty((B, Hq, D), device=partials.device, dtype=dtype)
    if out_lse is None:
        out_lse = torch.empty((B, Hq), device=partials.device, dtype=torch.float32)
    st = lib().ring_attn_merge(_ptr(partials), _ptr(part_lse), _ptr(out), _ptr(out_lse), B, Hq, P, D,
                               _dtype_code(out), _stream())
    _check(st, "ring_attn_merge")
    return out, out_lse


def ring_attn_decode(q, k, v, seqlens, P, scale=None, partials=None, part_lse=None, out=None, out_lse=None,
                     workspace=None):
    """Split-KV decode (per-chunk partials, then the merge).  Returns (out, out_lse)."""
    _cuda(q, k, v, seqlens, partials, part_lse, out, out_lse, workspace)
    B, Hq, Hkv, Smax, D = _decode_shapes(q, k, seqlens, P)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dev = q.device
    if partials is None:
        partials = torch.empty((B, Hq, P, D), device=dev, dtype=torch.float32)
    if part_lse is None:
        part_lse = torch.empty((B, Hq, P), device=dev, dtype=torch.float32)
    if out is None:
        out = torch.empty((B, Hq, D), device=dev, dtype=torch.bfloat16)
    if out_lse is None:
        out_lse = torch.empty((B, Hq), device=dev, dtype=torch.float32)
    if workspace is None:
        workspace = decode_workspace(B, Hq, Hkv, Smax, D, P, dev)
    st = lib().ring_attn_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(seqlens), _ptr(partials), _ptr(part_lse), _ptr(out),
                                _ptr(out_lse), B, Hq, Hkv, Smax, D, int(P), scale, _dtype_code(q), _ptr(workspace),
                                workspace.numel(), _stream())
    _check(st, "ring_attn_decode")
    return out, out_lse


def ring_attn_decode_fused(q, k, v, P, seqlens=None, shard_lens=None, scale=None, partials=None, part_lse=None,
                           out=None, out_lse=None, workspace=None):
    """Split-KV decode in one launch (partials plus the last-CTA merge).  Valid
    rows come from `seqlens` [B] (whole-cache lengths) or `shard_lens` [B,P]
    (per-chunk fill counts, e.g. after ring_attn_kv_append).  Returns (out, out_lse)."""
    if (seqlens is None) == (shard_lens is None):
        raise ValueError("give exactly one of seqlens / shard_lens")
    _cuda(q, k, v, seqlens, shard_lens, partials, part_lse, out, out_lse, workspace)
    B, Hq, D = q.shape
    _, Smax, Hkv, _ = k.shape
    lens = seqlens if seqlens is not None else shard_lens
    if lens.dtype != torch.int32 or lens.shape != ((B,) if seqlens is not None else (B, int(P))):
        raise ValueError("seqlens must be int32 [B], shard_lens int32 [B,P]")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    dev = q.device
    if partials is None:
        partials = torch.empty((B, Hq, P, D), device=dev, dtype=torch.float32)
    if part_lse is None:
        part_lse = torch.empty((B, Hq, P), device=dev, dtype=torch.float32)
    if out is None:
        out = torch.empty((B, Hq, D), device=dev, dtype=torch.bfloat16)
    if out_lse is None:
        out_lse = torch.empty((B, Hq), device=dev, dtype=torch.float32)
    if workspace is None:
        workspace = decode_workspace(B, Hq, Hkv, Smax, D, P, dev)
    st = lib().ring_attn_decode_fused(_ptr(q), _ptr(k), _ptr(v), _ptr(seqlens), _ptr(shard_lens), _ptr(partials),
                                      _ptr(part_lse), _ptr(out), _ptr(out_lse), B, Hq, Hkv, Smax, D, int(P), scale,
                                      _dtype_code(q), _ptr(workspace), workspace.numel(), _stream())
    _check(st, "ring_attn_decode_fused")
    return out, out_lse


def ring_attn_kv_append(k_cache, v_cache, k_new, v_new, shard_lens, n_appended, P, block):
    """Append k_new / v_new [B,T,Hkv,D] to the P-way sharded cache [B,Smax,Hkv,D],
    round-robin by blocks of `block` tokens; shard_lens [B,P] and n_appended [B]
    (int32, device) advance in place."""
    _cuda(k_cache, v_cache, k_new, v_new, shard_lens, n_appended)
    B, Smax, Hkv, D = k_cache.shape
    T = k_new.shape[1]
    if k_new.shape != (B, T, Hkv, D) or v_new.shape != k_new.shape or v_cache.shape != k_cache.shape:
        raise ValueError("k_new/v_new [B,T,Hkv,D] and caches [B,Smax,Hkv,D] expected")
    if k_new.dtype != k_cache.dtype or v_new.dtype != k_cache.dtype or v_cache.dtype != k_cache.dtype:
        raise ValueError("one dtype for caches and new tokens")
    if shard_lens.dtype != torch.int32 or shard_lens.shape != (B, int(P)):
        raise ValueError("shard_lens must be int32 [B,P]")
    if n_appended.dtype != torch.int32 or n_appended.shape != (B,):
        raise ValueError("n_appended must be int32 [B]")
    st = lib().ring_attn_kv_append(_ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new), _ptr(shard_lens),
                                   _ptr(n_appended), B, T, Hkv, Smax, D, int(P), int(block),
                                   _dtype_code(k_cache), _stream())
    _check(st, "ring_attn_kv_append")


# ---------------------------------------------------------------------------
# paged KV cache (layouts and rules: include/ring_attn.h)
# ---------------------------------------------------------------------------
def _one_device(*ts):
    """The index of the CUDA device all given tensors live on."""
    dev = -2
    for t in ts:
        if t is None:
            continue
        d = t.get_device()
        if d != dev:
            if d < 0:
                raise ValueError("tensors must live on a CUDA device")
            if dev >= 0:
                raise ValueError("tensors must live on one device")
            dev = d
    return dev


# current stream of a device as a plain integer (without making a Stream object, which costs 3 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


# RING_PAGE_EXTEND .. RING_PAGE_SELECT: the calls of ring_attn_paged_packed and their arguments' packing
_PACKED = {name: (i, struct.Struct(words), words.count("q") + words.count("d")) for i, (name, words) in enumerate((
    ("ring_attn_page_extend", "q" * 14), ("ring_attn_page_trim", "q" * 10), ("ring_attn_paged_append", "q" * 16),
    ("ring_attn_decode_paged", "q" * 23 + "d" + "q" * 4), ("ring_attn_page_bounds", "q" * 16),
    ("ring_attn_page_scores", "q" * 16), ("ring_attn_page_select", "q" * 11)))}


def _launch(name, dev, *args):
    """Call the library on the tensors' device, on that device's current torch stream."""
    call, words, n = _PACKED[name]
    fn = (_lib or lib()).ring_attn_paged_packed
    try:
        packed = words.pack(*args)
    except struct.error:
        raise ValueError(f"{name}: an argument is no 64-bit integer") from None
    if torch.cuda.current_device() == dev:
        st = fn(call, packed, n, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(call, packed, n, _raw_stream(dev))
    if st != RING_OK:
        _check(st, name)


def _int32(what, t, shape):
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous int32 {list(shape)}")
    return t.data_ptr()


def _table(block_table, B):
    """(pointer, W, row stride) of a block table [B, W] (rows may be slices of wider ones)."""
    if block_table.dim() == 2 and block_table.dtype == torch.int32:
        n, W = block_table.shape
        sn, s1 = block_table.stride()
        if n == B and (s1 == 1 or W == 1):
            return block_table.data_ptr(), W, sn if n > 1 else max(W, 1)
    raise ValueError("block_table must be int32 [B, W] with contiguous rows")


def _pool(k_pool, v_pool=None):
    """(num_pages, page_size, Hkv, D, page, token and head strides) of cache pools [num_pages, page_size, Hkv, D]."""
    strides = k_pool.stride()
    if len(strides) != 4 or strides[3] != 1:
        raise ValueError("pools must be [num_pages, page_size, Hkv, D] with contiguous last dimension")
    if v_pool is not None and (v_pool.shape != k_pool.shape or v_pool.stride() != strides or
                               v_pool.dtype != k_pool.dtype):
        raise ValueError("k_pool and v_pool must have one shape, dtype and strides")
    N, ps, Hkv, D = k_pool.shape
    sp, st, sh, _ = strides
    # the stride of a dimension of length 1 says nothing
    return N, ps, Hkv, D, (sp if N > 1 else ps * st), (st if ps > 1 else Hkv * D), (sh if Hkv > 1 else D)


def _rows3(what, x, shape, dtype):
    """(row stride, head stride) of x [n, heads, D] with contiguous D."""
    if x.shape == shape and x.dtype == dtype:
        sn, sh, s1 = x.stride()
        if s1 == 1:
            return (sn if shape[0] > 1 else shape[1] * shape[2]), (sh if shape[1] > 1 else shape[2])
    raise ValueError(f"{what} must be {list(shape)} of the cache's dtype with contiguous last dimension")


def ring_attn_page_extend(seq_lens, new_lens, block_table, free_pages, n_free, page_size, max_tokens=None,
                          slot_map=None, start_lens=None, cu_new=None):
    """Pages and cache rows for new_lens[b] new tokens of every sequence, on the
    device: seq_lens [B], block_table [B,W] and n_free [1] (pages on the free
    list free_pages) advance in place.  Returns (slot_map, start_lens, cu_new);
    slot_map has max_tokens entries (give one of the two), -1 past the call's
    tokens and for sequences that found no room (start_lens -1,
    ring_attn_device_error() RING_ECAPACITY)."""
    dev = _one_device(seq_lens, new_lens, block_table, free_pages, n_free, slot_map, start_lens, cu_new)
    B = seq_lens.numel()
    tp, W, ts = _table(block_table, B)
    if slot_map is None:
        if max_tokens is None:
            raise ValueError("give max_tokens or slot_map")
        slot_map = seq_lens.new_empty((int(max_tokens),), dtype=torch.int32)
    elif max_tokens is not None and slot_map.numel() != int(max_tokens):
        raise ValueError("slot_map must have max_tokens entries")
    if start_lens is None:
        start_lens = seq_lens.new_empty((B,), dtype=torch.int32)
    if cu_new is None:
        cu_new = seq_lens.new_empty((B + 1,), dtype=torch.int32)
    n, T = free_pages.numel(), slot_map.numel()
    _launch("ring_attn_page_extend", dev, _int32("seq_lens", seq_lens, (B,)), _int32("new_lens", new_lens, (B,)), tp,
            _int32("free_pages", free_pages, (n,)), _int32("n_free", n_free, (1,)),
            _int32("slot_map", slot_map, (T,)), _int32("start_lens", start_lens, (B,)),
            _int32("cu_new", cu_new, (B + 1,)), B, W, ts, int(page_size), n, T)
    return slot_map, start_lens, cu_new


def ring_attn_page_trim(seq_lens, keep_lens, block_table, free_pages, n_free, page_size):
    """Cut every sequence to keep_lens[b] tokens (0 ends it) and give the pages
    past its new end back to the free list, in place (negative table entries
    mark absent pages and are not given back)."""
    dev = _one_device(seq_lens, keep_lens, block_table, free_pages, n_free)
    B = seq_lens.numel()
    tp, W, ts = _table(block_table, B)
    n = free_pages.numel()
    _launch("ring_attn_page_trim", dev, _int32("seq_lens", seq_lens, (B,)), _int32("keep_lens", keep_lens, (B,)), tp,
            _int32("free_pages", free_pages, (n,)), _int32("n_free", n_free, (1,)), B, W, ts, int(page_size), n)


def ring_attn_paged_append(k_pool, v_pool, k_new, v_new, slot_map):
    """Write k_new / v_new [T,Hkv,D] into the rows slot_map [T] of the cache
    pools (slots outside the pools, -1 for instance, are skipped)."""
    dev = _one_device(k_pool, v_pool, k_new, v_new, slot_map)
    N, ps, Hkv, D, sp, st, sh = _pool(k_pool, v_pool)
    T = slot_map.numel()
    nt, nh = _rows3("k_new", k_new, (T, Hkv, D), k_pool.dtype)
    if _rows3("v_new", v_new, (T, Hkv, D), k_pool.dtype) != (nt, nh):
        raise ValueError("k_new and v_new must have the same strides")
    _launch("ring_attn_paged_append", dev, k_pool.data_ptr(), v_pool.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
            _int32("slot_map", slot_map, (T,)), T, Hkv, D, N, ps, sp, st, sh, nt, nh, _dtype_code(k_pool))


def ring_attn_decode_paged_workspace_bytes(D) -> int:
    return int(lib().ring_attn_decode_paged_workspace_bytes(int(D)))


def decode_paged_workspace(D, device="cuda"):
    """A zeroed workspace for ring_attn_decode_paged (one per stream; allocated with
    torch and zeroed on the current stream)."""
    n = ring_attn_decode_paged_workspace_bytes(D)
    if n == 0:
        raise ValueError("bad head dimension")
    return torch.zeros(n, device=device, dtype=torch.uint8)


def ring_attn_decode_paged(q, k_pool, v_pool, block_table, seq_lens, sel=None, n_sel=None, scale=None, out=None,
                           out_lse=None, workspace=None, out_dtype=None):
    """Attention of q [B,Hq,D] (one new token per sequence) over the seq_lens[b]
    keys of its cache pages, or over the pages sel [B,Hkv,K] / n_sel [B,Hkv]
    list for each kv head.  Returns (out, out_lse)."""
    dev = _one_device(q, k_pool, v_pool, block_table, seq_lens, sel, n_sel, out, out_lse, workspace)
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, D]")
    B, Hq, D = q.shape
    N, ps, Hkv, Dk, sp, st, sh = _pool(k_pool, v_pool)
    qb, qh = _rows3("q", q, (B, Hq, Dk), k_pool.dtype)
    tp, W, ts = _table(block_table, B)
    if (sel is None) != (n_sel is None):
        raise ValueError("give both sel and n_sel, or neither")
    K, selp, nselp = 0, 0, 0
    if sel is not None:
        K = sel.shape[-1] if sel.dim() else 0
        selp, nselp = _int32("sel", sel, (B, Hkv, K)), _int32("n_sel", n_sel, (B, Hkv))
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out is None:
        # (new_empty_strided takes two thirds of new_empty's time)
        out = q.new_empty_strided((B, Hq, D), (Hq * D, D, 1), dtype=out_dtype or q.dtype)
    elif tuple(out.shape) != (B, Hq, D) or not out.is_contiguous() or (out_dtype or out.dtype) != out.dtype:
        raise ValueError("out must be contiguous [B, Hq, D] of out_dtype")
    if out_lse is None:
        out_lse = q.new_empty_strided((B, Hq), (Hq, 1), dtype=torch.float32)
    elif tuple(out_lse.shape) != (B, Hq) or out_lse.dtype != torch.float32 or not out_lse.is_contiguous():
        raise ValueError("out_lse must be contiguous float32 [B, Hq]")
    if workspace is None:
        workspace = decode_paged_workspace(D, q.device)
    elif not workspace.is_contiguous():
        raise ValueError("tensors must be contiguous")
    _launch("ring_attn_decode_paged", dev, q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), tp,
            _int32("seq_lens", seq_lens, (B,)), selp, nselp, out.data_ptr(), out_lse.data_ptr(), B, Hq, Hkv, D, N, ps,
            W, K, qb, qh, sp, st, sh, ts, scale, _dtype_code(q), _dtype_code(out), workspace.data_ptr(),
            workspace.numel() * workspace.element_size())
    return out, out_lse


def ring_attn_page_bounds(k_pool, block_table, seq_lens, bounds=None, start_lens=None):
    """Minimum and maximum of the keys of every page, per kv head: bounds
    [num_pages,Hkv,2,D], brought up to date for the pages that hold tokens from
    start_lens[b] on (all pages without it; none of a sequence whose entry is
    negative).  Returns bounds."""
    dev = _one_device(k_pool, block_table, seq_lens, bounds, start_lens)
    N, ps, Hkv, D, sp, st, sh = _pool(k_pool)
    B = seq_lens.numel()
    tp, W, ts = _table(block_table, B)
    if bounds is None:
        bounds = k_pool.new_zeros((N, Hkv, 2, D))
    elif tuple(bounds.shape) != (N, Hkv, 2, D) or bounds.dtype != k_pool.dtype or not bounds.is_contiguous():
        raise ValueError("bounds must be contiguous [num_pages, Hkv, 2, D] of the cache's dtype")
    _launch("ring_attn_page_bounds", dev, k_pool.data_ptr(), bounds.data_ptr(), tp,
            _int32("seq_lens", seq_lens, (B,)),
            0 if start_lens is None else _int32("start_lens", start_lens, (B,)), B, Hkv, D, N, ps, W, sp, st, sh,
            ts, _dtype_code(k_pool))
    return bounds


def ring_attn_page_scores(q, bounds, block_table, seq_lens, page_size, scores=None):
    """scores [B,Hkv,W]: for every page an upper bound (up to float32 rounding) of
    q . k over its keys and the query heads of the kv head (-inf past the
    sequence's pages)."""
    dev = _one_device(q, bounds, block_table, seq_lens, scores)
    if q.dim() != 3 or bounds.dim() != 4 or bounds.shape[2] != 2 or not bounds.is_contiguous():
        raise ValueError("q [B, Hq, D] and contiguous bounds [num_pages, Hkv, 2, D] expected")
    B, Hq, _ = q.shape
    N, Hkv, _, D = bounds.shape
    qb, qh = _rows3("q", q, (B, Hq, D), bounds.dtype)
    tp, W, ts = _table(block_table, B)
    if scores is None:
        scores = q.new_empty((B, Hkv, W), dtype=torch.float32)
    elif tuple(scores.shape) != (B, Hkv, W) or scores.dtype != torch.float32 or not scores.is_contiguous():
        raise ValueError("scores must be contiguous float32 [B, Hkv, W]")
    _launch("ring_attn_page_scores", dev, q.data_ptr(), bounds.data_ptr(), tp, _int32("seq_lens", seq_lens, (B,)),
            scores.data_ptr(), B, Hq, Hkv, D, N, int(page_size), W, qb, qh, ts, _dtype_code(q))
    return scores


def ring_attn_page_select(scores, seq_lens, page_size, K, keep_first=1, keep_last=1, sel=None, n_sel=None):
    """The K best-scored pages per (sequence, kv head) of scores [B,Hkv,W], the
    first keep_first and last keep_last of the sequence always among them.
    Returns (sel [B,Hkv,K] ascending, then -1; n_sel [B,Hkv])."""
    dev = _one_device(scores, seq_lens, sel, n_sel)
    if scores.dim() != 3 or scores.dtype != torch.float32 or not scores.is_contiguous():
        raise ValueError("scores must be contiguous float32 [B, Hkv, W]")
    B, Hkv, W = scores.shape
    K = int(K)
    if sel is None:
        sel = seq_lens.new_empty_strided((B, Hkv, K), (Hkv * K, K, 1), dtype=torch.int32)
    if n_sel is None:
        n_sel = seq_lens.new_empty_strided((B, Hkv), (Hkv, 1), dtype=torch.int32)
    _launch("ring_attn_page_select", dev, scores.data_ptr(), _int32("seq_lens", seq_lens, (B,)),
            _int32("sel", sel, (B, Hkv, K)), _int32("n_sel", n_sel, (B, Hkv)), B, Hkv, W, int(page_size), K,
            int(keep_first), int(keep_last))
    return sel, n_sel


class RingAttnFunction(torch.autograd.Function):
    """Autograd over the whole ring: forward is ring_attn_fwd, backward is
    ring_attn_bwd on the saved q, k, v, out and lse.  Only marshalling: both
    passes run in the library's kernels."""

    @staticmethod
    def forward(ctx, q, k, v, P, causal=True, layout="zigzag", scale=None):
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()   # views (e.g. transposes) are copied once
        out, lse = ring_attn_fwd(q, k, v, P, causal, layout, scale)
        ctx.save_for_backward(q, k, v, out, lse)
        ctx.cfg = (P, causal, layout, scale)
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, out, lse = ctx.saved_tensors
        P, causal, layout, scale = ctx.cfg
        dq, dk, dv = ring_attn_bwd(q, k, v, out, lse, dout.to(q.dtype).contiguous(), P, causal, layout, scale)
        return dq, dk, dv, None, None, None, None


def ring_attention(q, k, v, P, causal=True, layout="zigzag", scale=None):
    """out = ring attention of q, k, v that autograd can differentiate
    (RingAttnFunction)."""
    return RingAttnFunction.apply(q, k, v, P, causal, layout, scale)


def ring_attn_sched_stats(S, P, causal, layout, tile_q=128, tile_k=128):
    """Host-side scheduler counts: (per_rank_pairs[P], full, partial, skipped)."""
    per = (ctypes.c_int64 * int(P))()
    f, pa, sk = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    st = lib().ring_attn_sched_stats(int(S), int(P), int(bool(causal)), _layout(layout), int(tile_q), int(tile_k),
                                     ctypes.cast(per, ctypes.c_void_p), ctypes.byref(f), ctypes.byref(pa),
                                     ctypes.byref(sk))
    _check(st, "ring_attn_sched_stats")
    return list(per), f.value, pa.value, sk.value


def ring_attn_selftest_wait(limit_us=1000):
    """Run the bounded-wait self test (see the header); check with ring_attn_device_error()."""
    _check(lib().ring_attn_selftest_wait(int(limit_us), _stream()), "ring_attn_selftest_wait")


def ring_attn_device_error():
    """Synchronise and return (status, site) of the device error words; what is
    reported is cleared (an expired wait first, lack of room by the next call)."""
    where = ctypes.c_int(0)
    st = lib().ring_attn_device_error(ctypes.byref(where))
    return st, where.value
