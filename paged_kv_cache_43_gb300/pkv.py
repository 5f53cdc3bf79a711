"""Thin ctypes binding of libpkv (include/pkv.h): argument marshalling only.

Every step of the path runs in the CUDA kernels behind the C ABI; this module
only checks tensor shapes/dtypes, fills the descriptor structs and passes data
pointers and the current CUDA stream.  If the library cannot be loaded the
calls raise: there is no fallback.
"""
from __future__ import annotations

import array
import ctypes
import os
import threading

import numpy as np
import torch

_lock = threading.Lock()
_lib = None

PKV_F32, PKV_BF16, PKV_FP8_E4M3, PKV_INT8 = 0, 1, 2, 3
# FP8 caches hold e4m3 codes; either dtype may carry them.
FP8_DTYPES = (torch.uint8, torch.float8_e4m3fn)
ERR_SLOT = 1 << 0
ERR_BLOCK_ID = 1 << 1
ERR_CONTEXT_LEN = 1 << 2
ERR_QUERY_LEN = 1 << 3
ERR_DECODE_QLEN = 1 << 4
ERR_TIMEOUT = 1 << 5
ERR_NONFINITE = 1 << 6
ERR_POSITION = 1 << 7
ERR_ACCEPTED = 1 << 8
EXPORTED = ("pkv_write", "pkv_write_fp8", "pkv_attention_workspace_size", "pkv_attention",
            "pkv_attention_fp8", "pkv_attention_static_scratch",
            "pkv_attention_cascade_workspace_size", "pkv_attention_cascade",
            "pkv_attention_cascade_fp8", "pkv_use_cascade",
            "pkv_write_int8", "pkv_attention_int8_workspace_size", "pkv_attention_int8",
            "pkv_copy_blocks",
            "pkv_rope_write", "pkv_rope_write_fp8", "pkv_rope",
            "pkv_attention_tree_workspace_size", "pkv_attention_tree", "pkv_attention_tree_fp8",
            "pkv_accept_drafts",
            "pkv_get_error", "pkv_status_string", "pkv_last_cuda_error",
            "pkv_last_cuda_error_string", "pkv_debug_wait_test")
STATIC_SCRATCH_BYTES = 64 << 20


class PkvError(RuntimeError):
    pass


class CacheDesc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_size", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class AttnMeta(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("num_tokens", ctypes.c_int32),
                ("num_q_heads", ctypes.c_int32), ("block_table_stride", ctypes.c_int32),
                ("max_query_len", ctypes.c_int32), ("max_context_len", ctypes.c_int32),
                ("num_decode_seqs", ctypes.c_int32), ("sliding_window", ctypes.c_int32),
                ("kv_split_tokens", ctypes.c_int32)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_size", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("max_position", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("q_out_stride", ctypes.c_int64),
                ("k_out_stride", ctypes.c_int64), ("eps", ctypes.c_float)]


def library_path() -> str:
    from . import build as _b
    return _b.LIB_PATH


def load(path: str | None = None):
    """Load libpkv.so (built by ``paged_kv_cache_43_gb300.build``)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = path or library_path()
        if not os.path.exists(path):
            raise PkvError(f"libpkv.so not built ({path}); run __graft_entry__.build()")
        lib = ctypes.CDLL(path)
        vp, i32, i64p = ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p
        lib.pkv_write.restype = ctypes.c_int
        lib.pkv_write.argtypes = [vp, vp, i64p, i32, vp, vp, ctypes.POINTER(CacheDesc), vp]
        lib.pkv_attention_workspace_size.restype = ctypes.c_size_t
        lib.pkv_attention_workspace_size.argtypes = [ctypes.POINTER(CacheDesc),
                                                     ctypes.POINTER(AttnMeta)]
        lib.pkv_attention.restype = ctypes.c_int
        lib.pkv_attention.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.c_float,
                                      ctypes.POINTER(CacheDesc), ctypes.POINTER(AttnMeta),
                                      vp, ctypes.c_size_t, vp]
        lib.pkv_write_fp8.restype = ctypes.c_int
        lib.pkv_write_fp8.argtypes = [vp, vp, i64p, i32, vp, vp, vp, vp,
                                      ctypes.POINTER(CacheDesc), vp]
        lib.pkv_attention_fp8.restype = ctypes.c_int
        lib.pkv_attention_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp,
                                          ctypes.POINTER(CacheDesc), ctypes.POINTER(AttnMeta),
                                          vp, ctypes.c_size_t, vp]
        lib.pkv_attention_cascade_workspace_size.restype = ctypes.c_size_t
        lib.pkv_attention_cascade_workspace_size.argtypes = [ctypes.POINTER(CacheDesc),
                                                             ctypes.POINTER(AttnMeta), i32]
        lib.pkv_attention_cascade.restype = ctypes.c_int
        lib.pkv_attention_cascade.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, i32,
                                              ctypes.POINTER(CacheDesc), ctypes.POINTER(AttnMeta),
                                              vp, ctypes.c_size_t, vp]
        lib.pkv_attention_cascade_fp8.restype = ctypes.c_int
        lib.pkv_attention_cascade_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, i32,
                                                  vp, vp, ctypes.POINTER(CacheDesc),
                                                  ctypes.POINTER(AttnMeta), vp, ctypes.c_size_t,
                                                  vp]
        lib.pkv_use_cascade.restype = ctypes.c_int
        lib.pkv_use_cascade.argtypes = [ctypes.POINTER(AttnMeta), i32]
        lib.pkv_attention_static_scratch.restype = ctypes.c_int
        lib.pkv_attention_static_scratch.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.c_float,
                                                     ctypes.POINTER(CacheDesc),
                                                     ctypes.POINTER(AttnMeta), vp]
        lib.pkv_write_int8.restype = ctypes.c_int
        lib.pkv_write_int8.argtypes = [vp] * 9 + [ctypes.POINTER(CacheDesc),
                                                  ctypes.POINTER(AttnMeta), vp]
        lib.pkv_attention_int8_workspace_size.restype = ctypes.c_size_t
        lib.pkv_attention_int8_workspace_size.argtypes = [ctypes.POINTER(CacheDesc),
                                                          ctypes.POINTER(AttnMeta)]
        lib.pkv_attention_int8.restype = ctypes.c_int
        lib.pkv_attention_int8.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp,
                                           ctypes.POINTER(CacheDesc), ctypes.POINTER(AttnMeta),
                                           vp, ctypes.c_size_t, vp]
        lib.pkv_copy_blocks.restype = ctypes.c_int
        lib.pkv_copy_blocks.argtypes = [vp, vp, i32, i32, vp, i32, vp]
        lib.pkv_rope_write.restype = ctypes.c_int
        lib.pkv_rope_write.argtypes = [vp] * 11 + [ctypes.POINTER(RopeDesc),
                                                   ctypes.POINTER(CacheDesc), vp]
        lib.pkv_rope_write_fp8.restype = ctypes.c_int
        lib.pkv_rope_write_fp8.argtypes = [vp] * 13 + [ctypes.POINTER(RopeDesc),
                                                       ctypes.POINTER(CacheDesc), vp]
        lib.pkv_rope.restype = ctypes.c_int
        lib.pkv_rope.argtypes = [vp] * 8 + [ctypes.POINTER(RopeDesc), vp]
        lib.pkv_attention_tree_workspace_size.restype = ctypes.c_size_t
        lib.pkv_attention_tree_workspace_size.argtypes = [ctypes.POINTER(CacheDesc),
                                                          ctypes.POINTER(AttnMeta)]
        lib.pkv_attention_tree.restype = ctypes.c_int
        lib.pkv_attention_tree.argtypes = [vp] * 8 + [ctypes.c_float, ctypes.POINTER(CacheDesc),
                                                      ctypes.POINTER(AttnMeta), vp,
                                                      ctypes.c_size_t, vp]
        lib.pkv_attention_tree_fp8.restype = ctypes.c_int
        lib.pkv_attention_tree_fp8.argtypes = [vp] * 8 + [ctypes.c_float, vp, vp,
                                                          ctypes.POINTER(CacheDesc),
                                                          ctypes.POINTER(AttnMeta), vp,
                                                          ctypes.c_size_t, vp]
        lib.pkv_accept_drafts.restype = ctypes.c_int
        lib.pkv_accept_drafts.argtypes = [vp, vp, i32, i32, vp, i32, vp, vp, i32, vp, vp, i32, vp,
                                          vp]
        lib.pkv_get_error.restype = ctypes.c_int
        lib.pkv_get_error.argtypes = [ctypes.POINTER(ctypes.c_int32), ctypes.c_int]
        lib.pkv_status_string.restype = ctypes.c_char_p
        lib.pkv_status_string.argtypes = [ctypes.c_int]
        lib.pkv_last_cuda_error.restype = ctypes.c_int
        lib.pkv_last_cuda_error.argtypes = []
        lib.pkv_last_cuda_error_string.restype = ctypes.c_char_p
        lib.pkv_last_cuda_error_string.argtypes = []
        lib.pkv_debug_wait_test.restype = ctypes.c_int
        lib.pkv_debug_wait_test.argtypes = [ctypes.c_int]
        _lib = lib
        return lib


def _check(status: int):
    if status != 0:
        lib = load()
        msg = f"pkv status {status}: {lib.pkv_status_string(status).decode()}"
        if status == -7:   # PKV_E_CUDA: say which CUDA error
            msg += f" ({lib.pkv_last_cuda_error_string().decode()})"
        raise PkvError(msg)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return PKV_BF16
    if t.dtype == torch.float32:
        return PKV_F32
    if t.dtype in FP8_DTYPES:
        return PKV_FP8_E4M3
    if t.dtype == torch.int8:
        return PKV_INT8
    raise PkvError(f"unsupported dtype {t.dtype}")


def _stream(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def cache_desc(k_cache: torch.Tensor) -> CacheDesc:
    nb, bs, hkv, d = k_cache.shape
    return CacheDesc(nb, bs, hkv, d, _dtype_code(k_cache))


def _require(t: torch.Tensor, name: str, dtype=None, ndim=None):
    if not t.is_cuda:
        raise PkvError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise PkvError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise PkvError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise PkvError(f"{name} must have {ndim} dims")


def write(k, v, slot_mapping, k_cache, v_cache, stream=None) -> None:
    """pkv_write: scatter k/v [T, Hkv, D] into the caches at slot_mapping[T]."""
    lib = load()
    for t, n in ((k, "k"), (v, "v"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _require(t, n, dtype=k_cache.dtype)
    _require(slot_mapping, "slot_mapping", dtype=torch.int64, ndim=1)
    T = slot_mapping.shape[0]
    if k.shape[0] < T or v.shape[0] < T:
        raise PkvError("k/v have fewer rows than slot_mapping")
    desc = cache_desc(k_cache)
    _check(lib.pkv_write(k.data_ptr(), v.data_ptr(), slot_mapping.data_ptr(), T,
                         k_cache.data_ptr(), v_cache.data_ptr(), ctypes.byref(desc),
                         _stream(stream)))


def write_fp8(k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale, stream=None) -> None:
    """pkv_write_fp8: quantise bf16 k/v [T, Hkv, D] with the per-kv-head
    scales (fp32 [Hkv]) into the e4m3 caches at slot_mapping[T]."""
    lib = load()
    for t, n in ((k, "k"), (v, "v")):
        _require(t, n, dtype=torch.bfloat16)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _require(t, n)
        if t.dtype not in FP8_DTYPES:
            raise PkvError(f"{n} must hold e4m3 codes (uint8 or float8_e4m3fn)")
    hkv = k_cache.shape[2]
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        _require(t, n, dtype=torch.float32, ndim=1)
        if t.shape[0] != hkv:
            raise PkvError(f"{n} must have num_kv_heads entries")
    _require(slot_mapping, "slot_mapping", dtype=torch.int64, ndim=1)
    T = slot_mapping.shape[0]
    if k.shape[0] < T or v.shape[0] < T:
        raise PkvError("k/v have fewer rows than slot_mapping")
    desc = cache_desc(k_cache)
    _check(lib.pkv_write_fp8(k.data_ptr(), v.data_ptr(), slot_mapping.data_ptr(), T,
                             k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                             v_scale.data_ptr(), ctypes.byref(desc), _stream(stream)))


def attn_meta(q, block_tables, context_lens, *, max_query_len, max_context_len,
              num_decode_seqs=-1, kv_split_tokens=0, sliding_window=0) -> AttnMeta:
    return AttnMeta(int(context_lens.shape[0]), int(q.shape[0]), int(q.shape[1]),
                    int(block_tables.shape[1]), int(max_query_len), int(max_context_len),
                    int(num_decode_seqs), int(sliding_window), int(kv_split_tokens))


def workspace_size(k_cache, meta: AttnMeta) -> int:
    desc = cache_desc(k_cache)
    n = load().pkv_attention_workspace_size(ctypes.byref(desc), ctypes.byref(meta))
    if n == ctypes.c_size_t(-1).value:
        raise PkvError("invalid attention description")
    return int(n)


def attention(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc, scale,
              *, max_query_len, max_context_len, num_decode_seqs=-1, kv_split_tokens=0,
              sliding_window=0, workspace=None, stream=None) -> None:
    """pkv_attention into ``out`` [T, Hq, D].  ``workspace`` (uint8 CUDA tensor)
    is allocated here when not given and the batch needs split-K scratch."""
    lib = load()
    for t, n in ((out, "out"), (q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _require(t, n, dtype=k_cache.dtype)
    _require(block_tables, "block_tables", dtype=torch.int32, ndim=2)
    _require(context_lens, "context_lens", dtype=torch.int32, ndim=1)
    _require(query_start_loc, "query_start_loc", dtype=torch.int32, ndim=1)
    if out.shape != q.shape:
        raise PkvError("out and q must have the same shape")
    meta = attn_meta(q, block_tables, context_lens, max_query_len=max_query_len,
                     max_context_len=max_context_len, num_decode_seqs=num_decode_seqs,
                     kv_split_tokens=kv_split_tokens, sliding_window=sliding_window)
    desc = cache_desc(k_cache)
    need = workspace_size(k_cache, meta)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else 0
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.pkv_attention(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(),
                             v_cache.data_ptr(), block_tables.data_ptr(),
                             context_lens.data_ptr(), query_start_loc.data_ptr(),
                             float(scale), ctypes.byref(desc), ctypes.byref(meta),
                             ws_ptr, ws_bytes, _stream(stream)))


def attention_fp8(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc, scale,
                  k_descale, v_descale, *, max_query_len, max_context_len, num_decode_seqs=-1,
                  kv_split_tokens=0, sliding_window=0, workspace=None, stream=None) -> None:
    """pkv_attention_fp8 into ``out`` [T, Hq, D] (bf16) over e4m3 caches;
    ``k_descale``/``v_descale`` fp32 [num_seqs, Hkv]."""
    lib = load()
    for t, n in ((out, "out"), (q, "q")):
        _require(t, n, dtype=torch.bfloat16)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _require(t, n)
        if t.dtype not in FP8_DTYPES:
            raise PkvError(f"{n} must hold e4m3 codes (uint8 or float8_e4m3fn)")
    _require(block_tables, "block_tables", dtype=torch.int32, ndim=2)
    _require(context_lens, "context_lens", dtype=torch.int32, ndim=1)
    _require(query_start_loc, "query_start_loc", dtype=torch.int32, ndim=1)
    for t, n in ((k_descale, "k_descale"), (v_descale, "v_descale")):
        _require(t, n, dtype=torch.float32, ndim=2)
        if tuple(t.shape) != (context_lens.shape[0], k_cache.shape[2]):
            raise PkvError(f"{n} must be [num_seqs, num_kv_heads]")
    if out.shape != q.shape:
        raise PkvError("out and q must have the same shape")
    meta = attn_meta(q, block_tables, context_lens, max_query_len=max_query_len,
                     max_context_len=max_context_len, num_decode_seqs=num_decode_seqs,
                     kv_split_tokens=kv_split_tokens, sliding_window=sliding_window)
    desc = cache_desc(k_cache)
    need = workspace_size(k_cache, meta)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else 0
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.pkv_attention_fp8(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(),
                                 v_cache.data_ptr(), block_tables.data_ptr(),
                                 context_lens.data_ptr(), query_start_loc.data_ptr(),
                                 float(scale), k_descale.data_ptr(), v_descale.data_ptr(),
                                 ctypes.byref(desc), ctypes.byref(meta), ws_ptr, ws_bytes,
                                 _stream(stream)))


def cascade_workspace_size(k_cache, meta: AttnMeta, common_prefix_blocks: int) -> int:
    desc = cache_desc(k_cache)
    n = load().pkv_attention_cascade_workspace_size(ctypes.byref(desc), ctypes.byref(meta),
                                                    int(common_prefix_blocks))
    if n == ctypes.c_size_t(-1).value:
        raise PkvError("invalid cascade description")
    return int(n)


def use_cascade(meta: AttnMeta, common_prefix_blocks: int) -> bool:
    """The cascade gate (>= 256 shared tokens, >= 8 sequences, no window,
    decode rows)."""
    return bool(load().pkv_use_cascade(ctypes.byref(meta), int(common_prefix_blocks)))


def attention_cascade(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc, scale,
                      common_prefix_blocks, *, max_context_len, max_query_len=1,
                      num_decode_seqs=-1, kv_split_tokens=0, workspace=None,
                      stream=None) -> None:
    """pkv_attention_cascade: a batch (decode rows, then chunked-prefill
    sequences) whose sequences share their first ``common_prefix_blocks``
    blocks; same result as attention()."""
    lib = load()
    for t, n in ((out, "out"), (q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _require(t, n, dtype=k_cache.dtype)
    _require(block_tables, "block_tables", dtype=torch.int32, ndim=2)
    _require(context_lens, "context_lens", dtype=torch.int32, ndim=1)
    _require(query_start_loc, "query_start_loc", dtype=torch.int32, ndim=1)
    meta = attn_meta(q, block_tables, context_lens, max_query_len=max_query_len,
                     max_context_len=max_context_len, num_decode_seqs=num_decode_seqs,
                     kv_split_tokens=kv_split_tokens)
    desc = cache_desc(k_cache)
    if workspace is None:
        need = cascade_workspace_size(k_cache, meta, common_prefix_blocks)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _check(lib.pkv_attention_cascade(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(),
                                     v_cache.data_ptr(), block_tables.data_ptr(),
                                     context_lens.data_ptr(), query_start_loc.data_ptr(),
                                     float(scale), int(common_prefix_blocks), ctypes.byref(desc),
                                     ctypes.byref(meta), workspace.data_ptr(),
                                     workspace.numel() * workspace.element_size(),
                                     _stream(stream)))


def attention_cascade_fp8(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                          scale, common_prefix_blocks, k_descale, v_descale, *, max_context_len,
                          max_query_len=1, num_decode_seqs=-1, kv_split_tokens=0,
                          workspace=None, stream=None) -> None:
    """pkv_attention_cascade_fp8: attention_cascade over e4m3 caches with the
    descales of attention_fp8."""
    lib = load()
    for t, n in ((out, "out"), (q, "q")):
        _require(t, n, dtype=torch.bfloat16)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _require(t, n)
        if t.dtype not in FP8_DTYPES:
            raise PkvError(f"{n} must hold e4m3 codes (uint8 or float8_e4m3fn)")
    _require(block_tables, "block_tables", dtype=torch.int32, ndim=2)
    _require(context_lens, "context_lens", dtype=torch.int32, ndim=1)
    _require(query_start_loc, "query_start_loc", dtype=torch.int32, ndim=1)
    for t, n in ((k_descale, "k_descale"), (v_descale, "v_descale")):
        _require(t, n, dtype=torch.float32, ndim=2)
        if tuple(t.shape) != (context_lens.shape[0], k_cache.shape[2]):
            raise PkvError(f"{n} must be [num_seqs, num_kv_heads]")
    meta = attn_meta(q, block_tables, context_lens, max_query_len=max_query_len,
                     max_context_len=max_context_len, num_decode_seqs=num_decode_seqs,
                     kv_split_tokens=kv_split_tokens)
    desc = cache_desc(k_cache)
    if workspace is None:
        need = cascade_workspace_size(k_cache, meta, common_prefix_blocks)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _check(lib.pkv_attention_cascade_fp8(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(),
                                         v_cache.data_ptr(), block_tables.data_ptr(),
                                         context_lens.data_ptr(), query_start_loc.data_ptr(),
                                         float(scale), int(common_prefix_blocks),
                                         k_descale.data_ptr(), v_descale.data_ptr(),
                                         ctypes.byref(desc), ctypes.byref(meta),
                                         workspace.data_ptr(),
                                         workspace.numel() * workspace.element_size(),
                                         _stream(stream)))


def attention_static_scratch(out, q, k_cache, v_cache, block_tables, context_lens,
                             query_start_loc, scale, *, max_query_len, max_context_len,
                             num_decode_seqs=-1, kv_split_tokens=0, sliding_window=0,
                             stream=None) -> int:
    """pkv_attention_static_scratch: pkv_attention with the split-K workspace
    taken from the library's own fixed device array (no allocation anywhere).
    Returns the C status (0 = enqueued; PKV_E_WORKSPACE = batch needs more than
    STATIC_SCRATCH_BYTES)."""
    lib = load()
    for t, n in ((out, "out"), (q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _require(t, n, dtype=k_cache.dtype)
    _require(block_tables, "block_tables", dtype=torch.int32, ndim=2)
    _require(context_lens, "context_lens", dtype=torch.int32, ndim=1)
    _require(query_start_loc, "query_start_loc", dtype=torch.int32, ndim=1)
    meta = attn_meta(q, block_tables, context_lens, max_query_len=max_query_len,
                     max_context_len=max_context_len, num_decode_seqs=num_decode_seqs,
                     kv_split_tokens=kv_split_tokens, sliding_window=sliding_window)
    desc = cache_desc(k_cache)
    return int(lib.pkv_attention_static_scratch(
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        block_tables.data_ptr(), context_lens.data_ptr(), query_start_loc.data_ptr(),
        float(scale), ctypes.byref(desc), ctypes.byref(meta), _stream(stream)))


_BF16, _I8, _I32, _F32, _U8 = (torch.bfloat16, torch.int8, torch.int32, torch.float32,
                               torch.uint8)
_NO_SIZE = ctypes.c_size_t(-1).value


def _int8_fits(dev: int, x, y, kc, vc, bt, cl, qsl, ks, vs) -> bool:
    """Whether an int8 call's tensors (rows x, y; caches; table, lengths, row
    starts; scales) are contiguous ones of their types on CUDA device `dev`
    whose shapes fit (_int8_batch says what does not).  One expression: a small
    decode step's kernel is over in microseconds, and each of these is 0.07."""
    c, r, n = kc.shape, x.shape, cl.shape
    return (x.dtype is _BF16 and y.dtype is _BF16 and kc.dtype is _I8 and vc.dtype is _I8
            and bt.dtype is _I32 and cl.dtype is _I32 and qsl.dtype is _I32
            and ks.dtype is _F32 and vs.dtype is _F32
            and (dev == x.get_device() == y.get_device() == kc.get_device() == vc.get_device()
                 == bt.get_device() == cl.get_device() == qsl.get_device() == ks.get_device()
                 == vs.get_device())
            and x.is_contiguous() and y.is_contiguous() and kc.is_contiguous()
            and vc.is_contiguous() and bt.is_contiguous() and cl.is_contiguous()
            and qsl.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()
            and len(c) == 4 and len(r) == 3 and len(n) == 1 and bt.dim() == 2 and qsl.dim() == 1
            and vc.shape == c and y.shape == r and r[2] == c[3]
            and ks.shape == vs.shape == (c[0], c[2])
            and bt.shape[0] >= n[0] and qsl.shape[0] > n[0])


def _refuse(dev: int, **tensors) -> None:
    """Says what is wrong with the first tensor (name=(tensor, dtype)) that
    _int8_fits did not take."""
    for name, (t, dtype) in tensors.items():
        _require(t, name, dtype=dtype)
        if t.get_device() != dev:
            raise PkvError(f"{name} must be on the current CUDA device ({dev})")


def _current_device() -> int:
    try:
        return torch.cuda.current_device()
    except (RuntimeError, AssertionError):   # no driver, or a torch without CUDA
        return -2                            # (no tensor is there)


def _int8_batch(dev, k_cache, v_cache, block_tables, context_lens, query_start_loc, k_scales,
                v_scales, **rows) -> None:
    """Checks the tensors of an int8 call one by one against each other (the
    rows bf16, by name); the calls make the same checks in one go first, since a
    decode step's kernel is over in microseconds."""
    bf16, i32, i8, f32 = torch.bfloat16, torch.int32, torch.int8, torch.float32
    _refuse(dev, **{n: (t, bf16) for n, t in rows.items()}, k_cache=(k_cache, i8),
            v_cache=(v_cache, i8), block_tables=(block_tables, i32),
            context_lens=(context_lens, i32), query_start_loc=(query_start_loc, i32),
            k_scales=(k_scales, f32), v_scales=(v_scales, f32))
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise PkvError("k_cache and v_cache must both be [num_blocks, 16, num_kv_heads, head_size]")
    for t, n in ((k_scales, "k_scales"), (v_scales, "v_scales")):
        if t.shape != (k_cache.shape[0], k_cache.shape[2]):
            raise PkvError(f"{n} must be [num_blocks, num_kv_heads]")
    if block_tables.dim() != 2 or context_lens.dim() != 1 or query_start_loc.dim() != 1 or \
            block_tables.shape[0] < context_lens.shape[0] or \
            query_start_loc.shape[0] < context_lens.shape[0] + 1:
        raise PkvError("block_tables [num_seqs, stride], context_lens [num_seqs] and "
                       "query_start_loc [num_seqs + 1] must fit together")
    one, two = rows.values()
    if one.dim() != 3 or one.shape != two.shape or one.shape[2] != k_cache.shape[3] or \
            ("k" in rows and one.shape[1] != k_cache.shape[2]):
        raise PkvError(" and ".join(rows) + " must both be [num_tokens, heads, head_size]")


def write_int8(k, v, block_tables, context_lens, query_start_loc, k_cache, v_cache, k_scales,
               v_scales, *, max_query_len, stream=None) -> None:
    """pkv_write_int8: the batch's bf16 rows k/v [T, Hkv, D] into the int8
    caches at the sequences' last positions, making the scales fp32
    [num_blocks, Hkv] of the blocks they touch."""
    lib = _lib or load()
    dev = _current_device()
    if not (_int8_fits(dev, k, v, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                       k_scales, v_scales) and k.shape[1] == k_cache.shape[2]):
        _int8_batch(dev, k_cache, v_cache, block_tables, context_lens, query_start_loc, k_scales,
                    v_scales, k=k, v=v)
    nb, bs, hkv, d = k_cache.shape
    desc = CacheDesc(nb, bs, hkv, d, PKV_INT8)
    meta = AttnMeta(context_lens.shape[0], k.shape[0], hkv, block_tables.shape[1], max_query_len,
                    0, -1, 0, 0)
    st = lib.pkv_write_int8(k.data_ptr(), v.data_ptr(), block_tables.data_ptr(),
                            context_lens.data_ptr(), query_start_loc.data_ptr(),
                            k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(),
                            v_scales.data_ptr(), desc, meta, _stream_on(dev, stream))
    if st != 0:
        _check(st)


# (the current stream's handle without the Stream object around it: 1 us of a
# call that takes 10)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_on(dev: int, stream) -> int:
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return (stream if stream is not None else torch.cuda.current_stream(dev)).cuda_stream


def workspace_size_int8(k_cache, meta: AttnMeta) -> int:
    desc = cache_desc(k_cache)
    n = load().pkv_attention_int8_workspace_size(desc, meta)
    if n == ctypes.c_size_t(-1).value:
        raise PkvError("invalid attention description")
    return int(n)


def attention_int8(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc, scale,
                   k_scales, v_scales, *, max_query_len, max_context_len, num_decode_seqs=-1,
                   kv_split_tokens=0, sliding_window=0, workspace=None, stream=None) -> None:
    """pkv_attention_int8 into ``out`` [T, Hq, D] (bf16) over int8 caches with
    the scales write_int8 made.  ``workspace`` (uint8 CUDA tensor of
    workspace_size_int8 bytes) is allocated here when not given and needed."""
    lib = _lib or load()
    dev = _current_device()
    if not _int8_fits(dev, out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                      k_scales, v_scales):
        _int8_batch(dev, k_cache, v_cache, block_tables, context_lens, query_start_loc, k_scales,
                    v_scales, out=out, q=q)
    nb, bs, hkv, d = k_cache.shape
    T, hq, _ = q.shape
    desc = CacheDesc(nb, bs, hkv, d, PKV_INT8)
    meta = AttnMeta(context_lens.shape[0], T, hq, block_tables.shape[1], max_query_len,
                    max_context_len, num_decode_seqs, sliding_window, kv_split_tokens)
    ws_ptr, ws_bytes = 0, 0
    if workspace is None:
        ws_bytes = lib.pkv_attention_int8_workspace_size(desc, meta)
        if ws_bytes == _NO_SIZE:
            ws_bytes = 0   # (the call itself says what is wrong)
        elif ws_bytes:
            if stream is None:
                workspace = q.new_empty(ws_bytes, dtype=_U8)
            else:          # scratch of the stream that uses it
                with torch.cuda.stream(stream):
                    workspace = q.new_empty(ws_bytes, dtype=_U8)
            ws_ptr = workspace.data_ptr()
    else:
        _refuse(dev, workspace=(workspace, None))
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.nbytes
    st = lib.pkv_attention_int8(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(),
                                v_cache.data_ptr(), block_tables.data_ptr(),
                                context_lens.data_ptr(), query_start_loc.data_ptr(), scale,
                                k_scales.data_ptr(), v_scales.data_ptr(), desc, meta, ws_ptr,
                                ws_bytes, _stream_on(dev, stream))
    if st != 0:
        _check(st)


def copy_blocks(buffers, pairs, stream=None) -> None:
    """pkv_copy_blocks: copies whole blocks of every buffer (CUDA tensors
    [num_blocks, ...]: the K and V caches and scales of all layers) along
    ``pairs`` (host ints [n, 2]: from, to), in order."""
    lib = _lib or load()
    pairs = np.asarray(pairs)
    if pairs.size == 0 or len(buffers) == 0:
        return
    if pairs.ndim != 2 or pairs.shape[1] != 2 or pairs.dtype.kind not in "iu":
        raise PkvError("pairs must be integers [n, 2] (from, to)")
    dev = _current_device()
    nb = buffers[0].shape[0] if buffers[0].dim() else 0
    if pairs.dtype != np.int32:
        if pairs.min() < 0 or pairs.max() >= nb:   # (before 32 bits cut them short)
            raise PkvError("pairs name a block that there is not")
        pairs = pairs.astype(np.int32)
    pairs = np.ascontiguousarray(pairs)
    for t in buffers:
        if t.get_device() != dev or not t.is_contiguous() or t.dim() == 0 or t.shape[0] != nb:
            _refuse(dev, buffers=(t, None))
            raise PkvError("buffers must all be [num_blocks, ...] of the same number of blocks")
    # (arrays of the C call: pointers and bytes of a page)
    ptrs = array.array("Q", [t.data_ptr() for t in buffers])
    page = array.array("q", [t.nbytes // nb for t in buffers] if nb else [0] * len(buffers))
    st = lib.pkv_copy_blocks(ptrs.buffer_info()[0], page.buffer_info()[0], len(buffers), nb,
                             pairs.ctypes.data, pairs.shape[0], _stream_on(dev, stream))
    if st != 0:
        _check(st)


# ---------------------------------------- steps with drafted tokens
#
# (Checked in one expression first, one by one only to say what is wrong: as the
# int8 calls.)

_I64 = torch.int64
_FP8 = frozenset(FP8_DTYPES)


def _rows_ok(t, dtype, shape, dev) -> bool:
    """Rows [tokens, heads, d] whose heads lie densely; tokens any stride apart."""
    return (t.dtype is dtype and t.get_device() == dev and t.shape == shape
            and (t.is_contiguous() or (t.stride(2) == 1 and (shape[1] == 1
                                                             or t.stride(1) == shape[2]))))


def _rope_desc(dev, q, k, v, q_out, k_out, positions, cos_sin, q_weight, k_weight, eps,
               interleaved) -> RopeDesc:
    """Checks the tensors of a rope call (v or k_out None) and describes them."""
    if q.dim() != 3 or k.dim() != 3:
        raise PkvError("q and k must be [num_tokens, heads, head_size]")
    dt, qs, ks = q.dtype, q.shape, k.shape
    tokens, hq, d = qs
    hkv = ks[1]
    if dt is not _BF16 and dt is not _F32:
        raise PkvError(f"unsupported dtype {dt}")
    other = k_out if v is None else v
    if not (_rows_ok(q, dt, qs, dev) and _rows_ok(k, dt, (tokens, hkv, d), dev)
            and _rows_ok(q_out, dt, qs, dev) and _rows_ok(other, dt, ks, dev)):
        for n, t, h in (("q", q, hq), ("k", k, hkv), ("q_out", q_out, hq),
                        ("v" if v is not None else "k_out", other, hkv)):
            if t.get_device() != dev:
                raise PkvError(f"{n} must be on the current CUDA device ({dev})")
            if not _rows_ok(t, dt, (tokens, h, d), dev):
                raise PkvError(f"{n} must be {dt} [{tokens}, {h}, {d}] with dense heads")
    cs = cos_sin.shape
    if not (positions.dtype is _I64 and cos_sin.dtype is _F32
            and positions.get_device() == dev == cos_sin.get_device()
            and positions.is_contiguous() and cos_sin.is_contiguous()
            and positions.shape == (tokens,) and len(cs) == 2):
        _refuse(dev, positions=(positions, _I64), cos_sin=(cos_sin, _F32))
        raise PkvError("positions must be [num_tokens], cos_sin [max_position, rot_dim]")
    for n, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and not (w.dtype is dt and w.shape == (d,) and w.get_device() == dev
                                  and w.is_contiguous()):
            _refuse(dev, **{n: (w, dt)})
            raise PkvError(f"{n} must be [{d}]")
    if tokens > 1:
        sq, sk, so, s2 = q.stride(0), k.stride(0), q_out.stride(0), other.stride(0)
    else:
        sq = so = hq * d
        sk = s2 = hkv * d
    return RopeDesc(tokens, hq, hkv, d, PKV_BF16 if dt is _BF16 else PKV_F32, cs[1], cs[0],
                    1 if interleaved else 0, sq, sk, s2, so, s2, eps)


def _rope_write(call, q_out, q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, scales,
                fp8, q_weight, k_weight, eps, interleaved, stream) -> None:
    dev = _current_device()
    desc = _rope_desc(dev, q, k, v, q_out, None, positions, cos_sin, q_weight, k_weight, eps,
                      interleaved)
    kd, c = k_cache.dtype, k_cache.shape
    if not ((kd in _FP8 if fp8 else kd is q.dtype) and v_cache.dtype is kd
            and slot_mapping.dtype is _I64
            and k_cache.get_device() == dev == v_cache.get_device() == slot_mapping.get_device()
            and k_cache.is_contiguous() and v_cache.is_contiguous()
            and slot_mapping.is_contiguous() and len(c) == 4 and v_cache.shape == c
            and c[2] == desc.num_kv_heads and c[3] == desc.head_size
            and slot_mapping.shape == positions.shape):
        if fp8 and (kd not in _FP8 or v_cache.dtype not in _FP8):
            raise PkvError("the caches must hold e4m3 codes (uint8 or float8_e4m3fn)")
        _refuse(dev, slot_mapping=(slot_mapping, _I64),
                k_cache=(k_cache, None if fp8 else q.dtype),
                v_cache=(v_cache, None if fp8 else q.dtype))
        raise PkvError("k_cache and v_cache must both be [num_blocks, 16, num_kv_heads, "
                       "head_size], slot_mapping [num_tokens]")
    for n, t in zip(("k_scale", "v_scale"), scales):
        if not (t.dtype is _F32 and t.shape == (c[2],) and t.get_device() == dev
                and t.is_contiguous()):
            _refuse(dev, **{n: (t, _F32)})
            raise PkvError(f"{n} must have num_kv_heads entries")
    cache = CacheDesc(c[0], c[1], c[2], c[3], PKV_FP8_E4M3 if fp8 else desc.dtype)
    st = call(q_out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), positions.data_ptr(),
              cos_sin.data_ptr(), 0 if q_weight is None else q_weight.data_ptr(),
              0 if k_weight is None else k_weight.data_ptr(), slot_mapping.data_ptr(),
              k_cache.data_ptr(), v_cache.data_ptr(), *[t.data_ptr() for t in scales], desc, cache,
              _stream_on(dev, stream))
    if st != 0:
        _check(st)


def rope_write(q_out, q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, *,
               q_weight=None, k_weight=None, eps=1e-6, interleaved=False, stream=None) -> None:
    """pkv_rope_write: norms of the query and key heads (where weights [D] are given),
    rotation by cos_sin (fp32 [max_position, rot_dim]) at positions (int64 [T]), q [T, Hq,
    D] to q_out, k and v [T, Hkv, D] to the caches at slot_mapping [T], in one pass.  q, k,
    v and q_out may be slices of a larger row (tokens any stride apart); q_out may be q."""
    _rope_write((_lib or load()).pkv_rope_write, q_out, q, k, v, positions, cos_sin, slot_mapping,
                k_cache, v_cache, (), False, q_weight, k_weight, eps, interleaved, stream)


def rope_write_fp8(q_out, q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, k_scale,
                   v_scale, *, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                   stream=None) -> None:
    """pkv_rope_write_fp8: rope_write of bf16 rows into e4m3 caches with the scales of
    write_fp8 (fp32 [Hkv])."""
    _rope_write((_lib or load()).pkv_rope_write_fp8, q_out, q, k, v, positions, cos_sin,
                slot_mapping, k_cache, v_cache, (k_scale, v_scale), True, q_weight, k_weight, eps,
                interleaved, stream)


def rope(q_out, k_out, q, k, positions, cos_sin, *, q_weight=None, k_weight=None, eps=1e-6,
         interleaved=False, stream=None) -> None:
    """pkv_rope: rope_write's q and k rows alone, k to k_out [T, Hkv, D] (which may be k), as
    write_int8 wants them."""
    lib = _lib or load()
    dev = _current_device()
    desc = _rope_desc(dev, q, k, None, q_out, k_out, positions, cos_sin, q_weight, k_weight, eps,
                      interleaved)
    st = lib.pkv_rope(q_out.data_ptr(), k_out.data_ptr(), q.data_ptr(), k.data_ptr(),
                      positions.data_ptr(), cos_sin.data_ptr(),
                      0 if q_weight is None else q_weight.data_ptr(),
                      0 if k_weight is None else k_weight.data_ptr(), desc,
                      _stream_on(dev, stream))
    if st != 0:
        _check(st)


def workspace_size_tree(k_cache, meta: AttnMeta) -> int:
    desc = cache_desc(k_cache)
    n = load().pkv_attention_tree_workspace_size(desc, meta)
    if n == _NO_SIZE:
        raise PkvError("invalid attention description")
    return int(n)


def _attention_tree(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                    tree_mask, scale, descales, fp8, max_query_len, max_context_len,
                    kv_split_tokens, workspace, stream) -> None:
    lib = _lib or load()
    dev = _current_device()
    kd, c, r, n = k_cache.dtype, k_cache.shape, q.shape, context_lens.shape
    if not ((kd in _FP8 and q.dtype is _BF16 if fp8 else
             (kd is _BF16 or kd is _F32) and q.dtype is kd)
            and v_cache.dtype is kd and out.dtype is q.dtype and block_tables.dtype is _I32
            and context_lens.dtype is _I32 and query_start_loc.dtype is _I32
            and tree_mask.dtype is _I64
            and (dev == q.get_device() == out.get_device() == k_cache.get_device()
                 == v_cache.get_device() == block_tables.get_device()
                 == context_lens.get_device() == query_start_loc.get_device()
                 == tree_mask.get_device())
            and q.is_contiguous() and out.is_contiguous() and k_cache.is_contiguous()
            and v_cache.is_contiguous() and block_tables.is_contiguous()
            and context_lens.is_contiguous() and query_start_loc.is_contiguous()
            and tree_mask.is_contiguous()
            and len(c) == 4 and len(r) == 3 and len(n) == 1 and block_tables.dim() == 2
            and query_start_loc.dim() == 1 and v_cache.shape == c and out.shape == r
            and r[2] == c[3] and block_tables.shape[0] >= n[0] and query_start_loc.shape[0] > n[0]
            and tree_mask.shape == (r[0], (max_query_len + 63) // 64)):
        if fp8 and (kd not in _FP8 or v_cache.dtype not in _FP8):
            raise PkvError("the caches must hold e4m3 codes (uint8 or float8_e4m3fn)")
        if not fp8 and kd not in (_BF16, _F32):
            raise PkvError(f"unsupported cache dtype {kd} (bf16 or fp32; e4m3: "
                           "attention_tree_fp8; int8 is not taken)")
        row = _BF16 if fp8 else kd
        _refuse(dev, out=(out, row), q=(q, row), k_cache=(k_cache, kd), v_cache=(v_cache, kd),
                block_tables=(block_tables, _I32), context_lens=(context_lens, _I32),
                query_start_loc=(query_start_loc, _I32), tree_mask=(tree_mask, _I64))
        if len(c) != 4 or v_cache.shape != c:
            raise PkvError("k_cache and v_cache must both be [num_blocks, 16, num_kv_heads, "
                           "head_size]")
        if len(r) != 3 or out.shape != r or r[2] != c[3]:
            raise PkvError("out and q must both be [num_tokens, heads, head_size]")
        if tree_mask.dim() != 2 or tree_mask.shape != (r[0], (max_query_len + 63) // 64):
            raise PkvError("tree_mask must be [num_tokens, ceil(max_query_len / 64)]")
        raise PkvError("block_tables [num_seqs, stride], context_lens [num_seqs] and "
                       "query_start_loc [num_seqs + 1] must fit together")
    for name, t in zip(("k_descale", "v_descale"), descales):
        if not (t.dtype is _F32 and t.shape == (n[0], c[2]) and t.get_device() == dev
                and t.is_contiguous()):
            _refuse(dev, **{name: (t, _F32)})
            raise PkvError(f"{name} must be [num_seqs, num_kv_heads]")
    desc = CacheDesc(*c, PKV_FP8_E4M3 if fp8 else (PKV_BF16 if kd is _BF16 else PKV_F32))
    meta = AttnMeta(n[0], r[0], r[1], block_tables.shape[1], max_query_len, max_context_len, -1, 0,
                    kv_split_tokens)
    ws_ptr, ws_bytes = 0, 0
    if workspace is None:
        ws_bytes = lib.pkv_attention_tree_workspace_size(desc, meta)
        if ws_bytes == _NO_SIZE:
            ws_bytes = 0   # (the call itself says what is wrong)
        elif ws_bytes:
            if stream is None:
                workspace = q.new_empty(ws_bytes, dtype=_U8)
            else:          # scratch of the stream that uses it
                with torch.cuda.stream(stream):
                    workspace = q.new_empty(ws_bytes, dtype=_U8)
            ws_ptr = workspace.data_ptr()
    else:
        _refuse(dev, workspace=(workspace, None))
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.nbytes
    rest = (desc, meta, ws_ptr, ws_bytes, _stream_on(dev, stream))
    call = lib.pkv_attention_tree_fp8 if fp8 else lib.pkv_attention_tree
    st = call(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
              block_tables.data_ptr(), context_lens.data_ptr(), query_start_loc.data_ptr(),
              tree_mask.data_ptr(), scale, *[t.data_ptr() for t in descales], *rest)
    if st != 0:
        _check(st)


def attention_tree(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                   tree_mask, scale, *, max_query_len, max_context_len, kv_split_tokens=0,
                   workspace=None, stream=None) -> None:
    """pkv_attention_tree into ``out`` [T, Hq, D]: a sequence's query rows are its drafted
    tokens, its last keys theirs; tree_mask (int64 [T, ceil(max_query_len / 64)]) has bit j
    of row i set where draft i sees draft j.  ``workspace`` (uint8 CUDA tensor of
    workspace_size_tree bytes) is allocated here when not given and needed."""
    _attention_tree(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                    tree_mask, scale, (), False, max_query_len, max_context_len, kv_split_tokens,
                    workspace, stream)


def attention_tree_fp8(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                       tree_mask, scale, k_descale, v_descale, *, max_query_len, max_context_len,
                       kv_split_tokens=0, workspace=None, stream=None) -> None:
    """pkv_attention_tree_fp8: attention_tree over e4m3 caches with the descales of
    attention_fp8 (fp32 [num_seqs, Hkv])."""
    _attention_tree(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                    tree_mask, scale, (k_descale, v_descale), True, max_query_len,
                    max_context_len, kv_split_tokens, workspace, stream)


def accept_drafts(buffers, block_tables, context_lens, query_start_loc, accepted, num_accepted, *,
                  new_context_lens=None, stream=None) -> None:
    """pkv_accept_drafts: in every buffer (CUDA tensors [num_blocks, 16, ...]: the K and V
    caches of all layers, not int8 ones), moves the rows of each sequence's accepted drafts
    (int32 [num_seqs, max_accepted], rising; num_accepted [num_seqs] of them) right behind
    the keys before its drafts; their number with these goes to ``new_context_lens``."""
    lib = _lib or load()
    dev = _current_device()
    n = context_lens.shape
    lens = context_lens if new_context_lens is None else new_context_lens
    if not (block_tables.dtype is _I32 and context_lens.dtype is _I32
            and query_start_loc.dtype is _I32 and accepted.dtype is _I32
            and num_accepted.dtype is _I32 and lens.dtype is _I32
            and (dev == block_tables.get_device() == context_lens.get_device()
                 == query_start_loc.get_device() == accepted.get_device()
                 == num_accepted.get_device() == lens.get_device())
            and block_tables.is_contiguous() and context_lens.is_contiguous()
            and query_start_loc.is_contiguous() and accepted.is_contiguous()
            and num_accepted.is_contiguous() and lens.is_contiguous()
            and len(n) == 1 and block_tables.dim() == 2 and query_start_loc.dim() == 1
            and accepted.dim() == 2 and block_tables.shape[0] >= n[0]
            and query_start_loc.shape[0] > n[0] and accepted.shape[0] == n[0]
            and num_accepted.shape == n == lens.shape):
        _refuse(dev, block_tables=(block_tables, _I32), context_lens=(context_lens, _I32),
                query_start_loc=(query_start_loc, _I32), accepted=(accepted, _I32),
                num_accepted=(num_accepted, _I32), new_context_lens=(lens, _I32))
        raise PkvError("block_tables [num_seqs, stride], context_lens, num_accepted and "
                       "new_context_lens [num_seqs], accepted [num_seqs, most] and "
                       "query_start_loc [num_seqs + 1] must fit together")
    if len(buffers):
        # (mostly all alike: then one row's bytes are all rows')
        t0 = buffers[0]
        shape, dtype = t0.shape, t0.dtype
        alike = (len(shape) >= 3 and shape[1] == 16 and dtype is not _I8
                 and all([t.shape == shape and t.dtype is dtype and t.is_contiguous()
                          and t.get_device() == dev for t in buffers]))
        nb = shape[0] if len(shape) else 0
        if not alike:
            for t in buffers:
                if (t.get_device() != dev or not t.is_contiguous() or t.dtype is _I8
                        or t.dim() < 3 or t.shape[0] != nb or t.shape[1] != 16):
                    _refuse(dev, buffers=(t, None))
                    raise PkvError("buffers must all be [num_blocks, 16, ...] of the same number "
                                   "of blocks, and not of an int8 cache")
        ptrs = array.array("Q", [t.data_ptr() for t in buffers])
        if nb == 0:
            rows = array.array("q", [4]) * len(buffers)
        elif alike:
            rows = array.array("q", [t0.nbytes // (16 * nb)]) * len(buffers)
        else:
            rows = array.array("q", [t.nbytes // (16 * nb) for t in buffers])
    else:
        nb, ptrs, rows = 0, array.array("Q"), array.array("q")
    st = lib.pkv_accept_drafts(ptrs.buffer_info()[0], rows.buffer_info()[0], len(buffers), nb,
                               block_tables.data_ptr(), block_tables.shape[1],
                               context_lens.data_ptr(), query_start_loc.data_ptr(), n[0],
                               accepted.data_ptr(), num_accepted.data_ptr(), accepted.shape[1],
                               0 if new_context_lens is None else lens.data_ptr(),
                               _stream_on(dev, stream))
    if st != 0:
        _check(st)


def get_error(clear: bool = True) -> int:
    """Device error word (PKV_ERR_* bits); synchronises the device."""
    bits = ctypes.c_int32(0)
    _check(load().pkv_get_error(ctypes.byref(bits), int(clear)))
    return int(bits.value)


def debug_wait_test(enable: bool) -> None:
    """Test hook of the timeout path (pkv_debug_wait_test): while enabled,
    decode and tcgen05 prefill launches wait at most 20 us and withhold their
    first key block, so their waits run out and PKV_ERR_TIMEOUT is set."""
    _check(load().pkv_debug_wait_test(1 if enable else 0))


def status_string(status: int) -> str:
    return load().pkv_status_string(status).decode()


def run_step(wl, out, workspace=None, kv_split_tokens=0, sliding_window=0, stream=None) -> None:
    """One pass of the hot path over a workload: the KV write of this step's
    tokens, then attention over the updated cache."""
    write(wl.k_new, wl.v_new, wl.slot_mapping, wl.k_cache, wl.v_cache, stream=stream)
    attention(out, wl.q, wl.k_cache, wl.v_cache, wl.block_tables, wl.context_lens,
              wl.query_start_loc, wl.scale, max_query_len=wl.max_query_len,
              max_context_len=wl.max_context_len, num_decode_seqs=wl.num_decode_seqs,
              kv_split_tokens=kv_split_tokens, sliding_window=sliding_window,
              workspace=workspace, stream=stream)
