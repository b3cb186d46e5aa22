"""Python binding of libpkv.so (include/pkv.h): argument marshalling only.

Each function takes torch tensors that already live on the GPU, checks their
dtype / layout / device, and passes raw device pointers, sizes and the current
CUDA stream to the C entry point of the same name.  Every step of the
computation runs in the library's CUDA kernels; there is no fallback of any kind:
if the shared library is missing or a call fails, an exception is raised.
"""

from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpkv.so")

PKV_OK = 0
PKV_ERR_ARG = -1
PKV_ERR_SHAPE = -2
PKV_ERR_WORKSPACE = -3
PKV_ERR_LAUNCH = -4
PKV_ERR_DEVICE_INDEX = -5
PKV_ERR_TIMEOUT = -6
PKV_DECODE_METADATA_READY = 1

_lock = threading.Lock()
_lib = None
_workspaces = {}
_stream_workspaces = {}
_KEPT_WORKSPACES = 64   # at most; the oldest goes when another stream needs one


class ScoreOptions(ctypes.Structure):
    """pkv_score_options of include/pkv.h."""

    _fields_ = [("softcap", ctypes.c_float), ("window", ctypes.c_int32),
                ("alibi_slopes", ctypes.c_void_p), ("first_keys", ctypes.c_void_p),
                ("prefix_lens", ctypes.c_void_p)]


class PkvError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status) if _lib else status}")


def load_library(path: str = LIB_PATH):
    """Load libpkv.so; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build the CUDA library first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(path)
        P, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                ctypes.c_float, ctypes.c_size_t)
        lib.kv_cache_store.argtypes = [P, P, i64, i64, P, P, P, i64, i32, i32, i32, i64, P]
        lib.kv_cache_store.restype = i32
        lib.kv_cache_copy_blocks.argtypes = [P, P, P, P, i32, i32, i32, i32, i64, P]
        lib.kv_cache_copy_blocks.restype = i32
        lib.paged_decode_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32, i32]
        lib.paged_decode_workspace_bytes.restype = sz
        lib.paged_decode_num_splits.argtypes = [i32, i32, i32, i32, i32, i32, i32]
        lib.paged_decode_num_splits.restype = i32
        lib.paged_decode_attention.argtypes = [P, P, P, P, P, P, i32, P, i32, i32, i32, i32,
                                               i32, i64, f32, P, sz, i32, P]
        lib.paged_decode_attention.restype = i32
        lib.paged_decode_attention_flags.argtypes = [P, P, P, P, P, P, i32, P, i32, i32, i32,
                                                     i32, i32, i64, f32, P, sz, i32,
                                                     ctypes.c_uint32, P]
        lib.paged_decode_attention_flags.restype = i32
        lib.paged_decode_shared_prefix_workspace_bytes.argtypes = [i32] * 8
        lib.paged_decode_shared_prefix_workspace_bytes.restype = sz
        lib.paged_decode_attention_shared_prefix.argtypes = [P, P, P, P, P, P, i32, P, i32, i32,
                                                             i32, i32, i32, i64, f32, i32, P,
                                                             sz, i32, P]
        lib.paged_decode_attention_shared_prefix.restype = i32
        lib.paged_decode_attention_noalloc.argtypes = [P, P, P, P, P, P, i32, P, i32, i32, i32,
                                                       i32, i32, i64, f32, i32, P]
        lib.paged_decode_attention_noalloc.restype = i32
        lib.paged_decode_multiquery_workspace_bytes.argtypes = [i32] * 8
        lib.paged_decode_multiquery_workspace_bytes.restype = sz
        lib.paged_decode_attention_multiquery.argtypes = [P, P, P, P, P, P, i32, P, i32, i32, i32,
                                                          i32, i32, i32, i64, f32, P, sz, i32, P]
        lib.paged_decode_attention_multiquery.restype = i32
        lib.paged_decode_attention_store.argtypes = [P, P, P, P, P, i64, i64, P, P, P, P, i32,
                                                     P, i32, i32, i32, i32, i32, i64, f32, P,
                                                     sz, i32, P]
        lib.paged_decode_attention_store.restype = i32
        lib.paged_decode_attention_fp8_store.argtypes = [P, P, P, P, P, i64, i64, P, P, P, P,
                                                         i32, P, i32, i32, i32, i32, i32, i64,
                                                         f32, f32, f32, P, sz, i32, P]
        lib.paged_decode_attention_fp8_store.restype = i32
        lib.kv_cache_store_fp8.argtypes = [P, P, i64, i64, P, P, P, i64, i32, i32, i32, i64,
                                           f32, f32, P]
        lib.kv_cache_store_fp8.restype = i32
        lib.paged_decode_attention_fp8.argtypes = [P, P, P, P, P, P, i32, P, i32, i32, i32, i32,
                                                   i32, i64, f32, f32, f32, P, sz, i32, P]
        lib.paged_decode_attention_fp8.restype = i32
        lib.paged_prefill_attention.argtypes = [P, P, P, P, P, P, i32, P, P, i32, i32, i32,
                                                i32, i32, i32, i32, i64, f32, P]
        lib.paged_prefill_attention.restype = i32
        opt = ctypes.POINTER(ScoreOptions)
        store = [P, P, P, P, i64, i64, i64, P, P, P, P, P, i64, i32, i32, P, P, f32, i64, i32,
                 i32, i32, i32, i64]
        lib.kv_cache_store_norm_rope.argtypes = [*store, P]
        lib.kv_cache_store_norm_rope.restype = i32
        lib.kv_cache_store_norm_rope_fp8.argtypes = [*store, f32, f32, P]
        lib.kv_cache_store_norm_rope_fp8.restype = i32
        lib.paged_decode_scored_workspace_bytes.argtypes = [i32] * 9
        lib.paged_decode_scored_workspace_bytes.restype = sz
        decode = [P, P, P, P, P, P, i32, P, i32, i32, i32, i32, i32, i64, f32]
        lib.paged_decode_attention_scored.argtypes = [*decode, opt, P, sz, i32, P]
        lib.paged_decode_attention_scored.restype = i32
        lib.paged_decode_attention_scored_fp8.argtypes = [*decode, f32, f32, opt, P, sz, i32, P]
        lib.paged_decode_attention_scored_fp8.restype = i32
        lib.paged_prefill_attention_scored.argtypes = [P, P, P, P, P, P, i32, P, P, i32, i64, i32,
                                                       i32, i32, i32, i32, i32, i64, f32, opt, P]
        lib.paged_prefill_attention_scored.restype = i32
        lib.pkv_get_device_error.argtypes = [P]
        lib.pkv_get_device_error.restype = i32
        lib.pkv_status_string.argtypes = [i32]
        lib.pkv_status_string.restype = ctypes.c_char_p
        lib.pkv_testing_set_wait_fault.argtypes = [i64, i32]
        lib.pkv_testing_set_wait_fault.restype = i32
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load_library().pkv_status_string(int(status)).decode()


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ptr(t: Optional[torch.Tensor]) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _need(t: torch.Tensor, name: str, dtype, ndim: Optional[int] = None,
          contiguous: bool = True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _pool_dims(k_cache: torch.Tensor, v_cache: torch.Tensor):
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    if k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    NB, bs, Hkv, D = k_cache.shape
    return NB, bs, Hkv, D


def _check(status: int, what: str):
    if status != PKV_OK:
        raise PkvError(status, what)


def kv_cache_store(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, slot_mapping: torch.Tensor, stream=None) -> None:
    """k, v: bf16 [T, Hkv, D] (each token's [Hkv, D] contiguous; token stride
    free); caches [NB, bs, Hkv, D]; slot_mapping int32 [T]."""
    lib = load_library()
    NB, bs, Hkv, D = _pool_dims(k_cache, v_cache)
    for name, t in (("k", k), ("v", v)):
        _need(t, name, torch.bfloat16, 3, contiguous=False)
        if tuple(t.shape[1:]) != (Hkv, D) or t.stride(2) != 1 or t.stride(1) != D:
            raise ValueError(f"{name} must be [T, {Hkv}, {D}] with contiguous rows")
    _need(slot_mapping, "slot_mapping", torch.int32, 1)
    T = k.shape[0]
    if v.shape[0] != T or slot_mapping.shape[0] != T:
        raise ValueError("k, v and slot_mapping disagree on T")
    _check(lib.kv_cache_store(_ptr(k), _ptr(v), k.stride(0), v.stride(0), _ptr(k_cache),
                              _ptr(v_cache), _ptr(slot_mapping), T, Hkv, D, bs, NB,
                              _stream(stream)), "kv_cache_store")


def kv_cache_copy_blocks(k_cache: torch.Tensor, v_cache: torch.Tensor,
                         src_blocks: torch.Tensor, dst_blocks: torch.Tensor,
                         stream=None) -> None:
    """Copy-on-write copies: block dst_blocks[i] of both caches becomes a copy
    of block src_blocks[i] (int32 device tensors of equal length)."""
    lib = load_library()
    NB, bs, Hkv, D = _pool_dims(k_cache, v_cache)
    _need(src_blocks, "src_blocks", torch.int32, 1)
    _need(dst_blocks, "dst_blocks", torch.int32, 1)
    if src_blocks.shape != dst_blocks.shape:
        raise ValueError("src_blocks and dst_blocks differ in length")
    _check(lib.kv_cache_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(src_blocks),
                                    _ptr(dst_blocks), src_blocks.shape[0], Hkv, D, bs, NB,
                                    _stream(stream)), "kv_cache_copy_blocks")


def paged_decode_workspace_bytes(B: int, Hq: int, Hkv: int, D: int, max_blocks_per_seq: int,
                                 block_size: int = 256, num_splits: int = 0) -> int:
    return int(load_library().paged_decode_workspace_bytes(B, Hq, Hkv, D, max_blocks_per_seq,
                                                           block_size, num_splits))


def paged_decode_num_splits(B: int, Hq: int, Hkv: int, D: int, max_blocks_per_seq: int,
                            block_size: int = 256, num_splits: int = 0) -> int:
    n = load_library().paged_decode_num_splits(B, Hq, Hkv, D, max_blocks_per_seq, block_size,
                                               num_splits)
    _check(min(n, 0), "paged_decode_num_splits")
    return int(n)


def decode_workspace(nbytes: int, device) -> torch.Tensor:
    """A zero-initialised, 256-byte aligned workspace of at least nbytes on
    `device`, reused across calls on that device (the library leaves its
    counters zeroed).  Callers running decode concurrently on several streams
    must pass their own workspaces instead."""
    dev = torch.device(device)
    key = (dev.type, dev.index if dev.index is not None else torch.cuda.current_device())
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=dev)
        _workspaces[key] = ws
    return ws


def paged_decode_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           block_tables: torch.Tensor, context_lens: torch.Tensor,
                           scale: float, out: Optional[torch.Tensor] = None,
                           lse: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, num_splits: int = 0,
                           want_lse: bool = True, stream=None, metadata_ready: bool = False
                           ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """q bf16 [B, Hq, D]; block_tables int32 [B, max_blocks]; context_lens int32
    [B].  Returns (out bf16 [B, Hq, D], lse fp32 [B, Hq] or None).
    metadata_ready: block_tables and context_lens were written before the
    stream's previous kernel started and no running kernel writes them
    (PKV_DECODE_METADATA_READY of paged_decode_attention_flags)."""
    lib = load_library()
    NB, bs, Hkv, D = _pool_dims(k_cache, v_cache)
    _need(q, "q", torch.bfloat16, 3)
    B, Hq, Dq = q.shape
    if Dq != D:
        raise ValueError("q head_dim differs from the cache's")
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    if block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("block_tables / context_lens batch differs from q")
    maxblk = block_tables.shape[1]
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, 3)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
    need = paged_decode_workspace_bytes(B, Hq, Hkv, D, maxblk, bs, num_splits)
    if workspace is None and need:
        workspace = decode_workspace(need, q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if metadata_ready:
        _check(lib.paged_decode_attention_flags(
            _ptr(out), _ptr(lse), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
            maxblk, _ptr(context_lens), B, Hq, Hkv, D, bs, NB, float(scale), _ptr(workspace),
            ws_bytes, int(num_splits), PKV_DECODE_METADATA_READY, _stream(stream)),
            "paged_decode_attention_flags")
        return out, lse
    _check(lib.paged_decode_attention(_ptr(out), _ptr(lse), _ptr(q), _ptr(k_cache),
                                      _ptr(v_cache), _ptr(block_tables), maxblk,
                                      _ptr(context_lens), B, Hq, Hkv, D, bs, NB, float(scale),
                                      _ptr(workspace), ws_bytes, int(num_splits),
                                      _stream(stream)), "paged_decode_attention")
    return out, lse


def paged_decode_attention_store(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                                 slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                                 v_cache: torch.Tensor, block_tables: torch.Tensor,
                                 context_lens: torch.Tensor, scale: float,
                                 out: Optional[torch.Tensor] = None,
                                 lse: Optional[torch.Tensor] = None,
                                 workspace: Optional[torch.Tensor] = None, num_splits: int = 0,
                                 want_lse: bool = True, stream=None
                                 ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Store the step's new tokens (k_new / v_new bf16 [B, Hkv, D] at
    slot_mapping[b], which must be -1 or the slot of position
    context_lens[b] - 1) and decode, in one launch.  Returns (out, lse) as
    paged_decode_attention."""
    lib = load_library()
    NB, bs, Hkv, D = _pool_dims(k_cache, v_cache)
    _need(q, "q", torch.bfloat16, 3)
    B, Hq, Dq = q.shape
    if Dq != D:
        raise ValueError("q head_dim differs from the cache's")
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        _need(t, name, torch.bfloat16, 3, contiguous=False)
        if tuple(t.shape) != (B, Hkv, D) or t.stride(2) != 1 or t.stride(1) != D:
            raise ValueError(f"{name} must be [B, {Hkv}, {D}] with contiguous rows")
    _need(slot_mapping, "slot_mapping", torch.int32, 1)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    maxblk = block_tables.shape[1]
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    need = paged_decode_workspace_bytes(B, Hq, Hkv, D, maxblk, bs, num_splits)
    if workspace is None and need:
        workspace = decode_workspace(need, q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.paged_decode_attention_store(
        _ptr(out), _ptr(lse), _ptr(q), _ptr(k_new), _ptr(v_new), k_new.stride(0),
        v_new.stride(0), _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
        maxblk, _ptr(context_lens), B, Hq, Hkv, D, bs, NB, float(scale), _ptr(workspace),
        ws_bytes, int(num_splits), _stream(stream)), "paged_decode_attention_store")
    return out, lse


def _fp8_pool_dims(k_cache: torch.Tensor, v_cache: torch.Tensor):
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _need(t, name, torch.uint8, 4)
    if k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    NB, bs, Hkv, D = k_cache.shape
    return NB, bs, Hkv, D


def kv_cache_store_fp8(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                       v_cache: torch.Tensor, slot_mapping: torch.Tensor, k_scale: float,
                       v_scale: float, stream=None) -> None:
    """Store bf16 k/v [T, Hkv, D] into uint8 E4M3 pools [NB, bs, Hkv, D] (one
    scale per tensor)."""
    lib = load_library()
    NB, bs, Hkv, D = _fp8_pool_dims(k_cache, v_cache)
    for name, t in (("k", k), ("v", v)):
        _need(t, name, torch.bfloat16, 3, contiguous=False)
        if t.stride(2) != 1 or t.stride(1) != D:
            raise ValueError(f"{name}: each token's [Hkv, D] rows must be contiguous")
    _need(slot_mapping, "slot_mapping", torch.int32, 1)
    T = k.shape[0]
    _check(lib.kv_cache_store_fp8(_ptr(k), _ptr(v), k.stride(0), v.stride(0), _ptr(k_cache),
                                  _ptr(v_cache), _ptr(slot_mapping), T, Hkv, D, bs, NB,
                                  float(k_scale), float(v_scale), _stream(stream)),
           "kv_cache_store_fp8")


def paged_decode_attention_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                               block_tables: torch.Tensor, context_lens: torch.Tensor,
                               scale: float, k_scale: float, v_scale: float,
                               out: Optional[torch.Tensor] = None,
                               lse: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None, num_splits: int = 0,
                               want_lse: bool = True, stream=None
                               ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Decode over uint8 E4M3 pools; q bf16 [B, Hq, D].  Returns (out bf16
    [B, Hq, D], lse fp32 [B, Hq] or None)."""
    lib = load_library()
    NB, bs, Hkv, D = _fp8_pool_dims(k_cache, v_cache)
    _need(q, "q", torch.bfloat16, 3)
    B, Hq, Dq = q.shape
    if Dq != D:
        raise ValueError("q head_dim differs from the cache's")
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    maxblk = block_tables.shape[1]
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    need = paged_decode_workspace_bytes(B, Hq, Hkv, D, maxblk, bs, num_splits)
    if workspace is None and need:
        workspace = decode_workspace(need, q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.paged_decode_attention_fp8(
        _ptr(out), _ptr(lse), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), maxblk,
        _ptr(context_lens), B, Hq, Hkv, D, bs, NB, float(scale), float(k_scale), float(v_scale),
        _ptr(workspace), ws_bytes, int(num_splits), _stream(stream)),
        "paged_decode_attention_fp8")
    return out, lse


def paged_decode_attention_fp8_store(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                                     slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                                     v_cache: torch.Tensor, block_tables: torch.Tensor,
                                     context_lens: torch.Tensor, scale: float, k_scale: float,
                                     v_scale: float, out: Optional[torch.Tensor] = None,
                                     lse: Optional[torch.Tensor] = None,
                                     workspace: Optional[torch.Tensor] = None,
                                     num_splits: int = 0, want_lse: bool = True, stream=None
                                     ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """kv_cache_store_fp8 of the new tokens (bf16 [B, Hkv, D], slot_mapping[b]
    -1 or the slot of position context_lens[b] - 1) and the E4M3 decode, in
    one launch.  Returns (out, lse) as paged_decode_attention_fp8."""
    lib = load_library()
    NB, bs, Hkv, D = _fp8_pool_dims(k_cache, v_cache)
    _need(q, "q", torch.bfloat16, 3)
    B, Hq, Dq = q.shape
    if Dq != D:
        raise ValueError("q head_dim differs from the cache's")
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        _need(t, name, torch.bfloat16, 3, contiguous=False)
        if tuple(t.shape) != (B, Hkv, D) or t.stride(2) != 1 or t.stride(1) != D:
            raise ValueError(f"{name} must be [B, {Hkv}, {D}] with contiguous rows")
    _need(slot_mapping, "slot_mapping", torch.int32, 1)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    maxblk = block_tables.shape[1]
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    need = paged_decode_workspace_bytes(B, Hq, Hkv, D, maxblk, bs, num_splits)
    if workspace is None and need:
        workspace = decode_workspace(need, q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.paged_decode_attention_fp8_store(
        _ptr(out), _ptr(lse), _ptr(q), _ptr(k_new), _ptr(v_new), k_new.stride(0),
        v_new.stride(0), _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
        maxblk, _ptr(context_lens), B, Hq, Hkv, D, bs, NB, float(scale), float(k_scale),
        float(v_scale), _ptr(workspace), ws_bytes, int(num_splits), _stream(stream)),
        "paged_decode_attention_fp8_store")
    return out, lse


def paged_decode_multiquery_workspace_bytes(B: int, q_len: int, Hq: int, Hkv: int, D: int,
                                            max_blocks_per_seq: int, block_size: int = 256,
                                            num_splits: int = 0) -> int:
    return int(load_library().paged_decode_multiquery_workspace_bytes(
        B, q_len, Hq, Hkv, D, max_blocks_per_seq, block_size, num_splits))


def paged_decode_attention_multiquery(q: torch.Tensor, k_cache: torch.Tensor,
                                      v_cache: torch.Tensor, block_tables: torch.Tensor,
                                      context_lens: torch.Tensor, scale: float,
                                      out: Optional[torch.Tensor] = None,
                                      lse: Optional[torch.Tensor] = None,
                                      workspace: Optional[torch.Tensor] = None,
                                      num_splits: int = 0, want_lse: bool = True, stream=None
                                      ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """q bf16 [B, q_len, Hq, D]: q_len new positions per sequence (already stored
    in the cache, counted in context_lens).  Returns (out bf16 [B, q_len, Hq, D],
    lse fp32 [B, q_len, Hq] or None)."""
    lib = load_library()
    NB, bs, Hkv, D = _pool_dims(k_cache, v_cache)
    _need(q, "q", torch.bfloat16, 4)
    B, q_len, Hq, Dq = q.shape
    if Dq != D:
        raise ValueError("q head_dim differs from the cache's")
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    if block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("block_tables / context_lens batch differs from q")
    maxblk = block_tables.shape[1]
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, 4)
    if lse is None and want_lse:
        lse = torch.empty((B, q_len, Hq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, 3)
    need = paged_decode_multiquery_workspace_bytes(B, q_len, Hq, Hkv, D, maxblk, bs, num_splits)
    if workspace is None and need:
        workspace = decode_workspace(need, q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.paged_decode_attention_multiquery(
        _ptr(out), _ptr(lse), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), maxblk,
        _ptr(context_lens), B, q_len, Hq, Hkv, D, bs, NB, float(scale), _ptr(workspace), ws_bytes,
        int(num_splits), _stream(stream)), "paged_decode_attention_multiquery")
    return out, lse


def paged_decode_shared_prefix_workspace_bytes(B: int, Hq: int, Hkv: int, D: int,
                                               max_blocks_per_seq: int,
                                               shared_prefix_tokens: int,
                                               block_size: int = 256,
                                               num_splits: int = 0) -> int:
    return int(load_library().paged_decode_shared_prefix_workspace_bytes(
        B, Hq, Hkv, D, max_blocks_per_seq, block_size, shared_prefix_tokens, num_splits))


def paged_decode_attention_shared_prefix(q: torch.Tensor, k_cache: torch.Tensor,
                                         v_cache: torch.Tensor, block_tables: torch.Tensor,
                                         context_lens: torch.Tensor, scale: float,
                                         shared_prefix_tokens: int,
                                         out: Optional[torch.Tensor] = None,
                                         lse: Optional[torch.Tensor] = None,
                                         workspace: Optional[torch.Tensor] = None,
                                         num_splits: int = 0, want_lse: bool = True,
                                         stream=None
                                         ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Decode for a batch whose sequences all start with the same
    `shared_prefix_tokens` tokens (the same physical blocks at the start of every
    table row).  Same results as paged_decode_attention."""
    lib = load_library()
    NB, bs, Hkv, D = _pool_dims(k_cache, v_cache)
    _need(q, "q", torch.bfloat16, 3)
    B, Hq, _ = q.shape
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    maxblk = block_tables.shape[1]
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, 3)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
    need = paged_decode_shared_prefix_workspace_bytes(B, Hq, Hkv, D, maxblk,
                                                      shared_prefix_tokens, bs, num_splits)
    if workspace is None and need:
        workspace = decode_workspace(need, q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.paged_decode_attention_shared_prefix(
        _ptr(out), _ptr(lse), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), maxblk,
        _ptr(context_lens), B, Hq, Hkv, D, bs, NB, float(scale), int(shared_prefix_tokens),
        _ptr(workspace), ws_bytes, int(num_splits), _stream(stream)),
        "paged_decode_attention_shared_prefix")
    return out, lse


NOALLOC_SCRATCH_BYTES = 16 << 20


def paged_decode_attention_noalloc(q: torch.Tensor, k_cache: torch.Tensor,
                                   v_cache: torch.Tensor, block_tables: torch.Tensor,
                                   context_lens: torch.Tensor, scale: float,
                                   out: torch.Tensor, lse: Optional[torch.Tensor] = None,
                                   num_splits: int = 0, stream=None) -> None:
    """Decode attention for callers that cannot allocate device memory: the
    split scratch is a fixed 16 MiB array inside the library instead of a
    caller-provided workspace, and the caller passes `out` (and optionally
    `lse`) already allocated.  Calls that overlap on the GPU race on that array."""
    lib = load_library()
    NB, bs, Hkv, D = _pool_dims(k_cache, v_cache)
    _need(q, "q", torch.bfloat16, 3)
    B, Hq, _ = q.shape
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    _need(out, "out", torch.bfloat16, 3)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
    _check(lib.paged_decode_attention_noalloc(
        _ptr(out), _ptr(lse), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
        block_tables.shape[1], _ptr(context_lens), B, Hq, Hkv, D, bs, NB, float(scale),
        int(num_splits), _stream(stream)), "paged_decode_attention_noalloc")


def paged_prefill_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            block_tables: torch.Tensor, cu_seqlens_q: torch.Tensor,
                            cu_seqlens_k: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int,
                            scale: float, out: Optional[torch.Tensor] = None,
                            lse: Optional[torch.Tensor] = None, want_lse: bool = True,
                            stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """q bf16 [sum Lq, Hq, D]; cu_seqlens int32 [B+1].  The new tokens' K/V must
    already be stored in the pool.  Returns (out bf16 [sum Lq, Hq, D], lse fp32
    [sum Lq, Hq] or None)."""
    lib = load_library()
    NB, bs, Hkv, D = _pool_dims(k_cache, v_cache)
    _need(q, "q", torch.bfloat16, 3)
    Nq, Hq, Dq = q.shape
    if Dq != D:
        raise ValueError("q head_dim differs from the cache's")
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    B = cu_seqlens_q.shape[0] - 1
    if cu_seqlens_k.shape[0] != B + 1 or block_tables.shape[0] != B:
        raise ValueError("cu_seqlens / block_tables batch sizes differ")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, 3)
    if lse is None and want_lse:
        lse = torch.empty((Nq, Hq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
    _check(lib.paged_prefill_attention(_ptr(out), _ptr(lse), _ptr(q), _ptr(k_cache),
                                       _ptr(v_cache), _ptr(block_tables),
                                       block_tables.shape[1], _ptr(cu_seqlens_q),
                                       _ptr(cu_seqlens_k), B, int(max_seqlen_q),
                                       int(max_seqlen_k), Hq, Hkv, D, bs, NB, float(scale),
                                       _stream(stream)), "paged_prefill_attention")
    return out, lse


class _Launch:
    """Makes the device of a call's tensors current, and the given stream (a torch
    stream or a raw handle), so that what the call allocates belongs to both."""

    def __init__(self, device: torch.device, stream):
        if device.type != "cuda":
            raise ValueError(f"the tensors must be on a CUDA device, not {device}")
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
                      else torch.cuda.default_stream(device))
        if stream is not None and stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        self._guards = [torch.cuda.device(device)]
        if stream is not None:
            self._guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self._guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self._guards):
            g.__exit__(*exc)
        return False


# The current device and its current stream as plain numbers (the public calls
# build a stream object each time: 3 us of a small call's 15).
def _current_device() -> int:
    return torch._C._cuda_getDevice()


def _current_stream(device_index: int) -> int:
    return torch._C._cuda_getCurrentRawStream(device_index)


def _workspace(given: Optional[torch.Tensor], nbytes: int, like: torch.Tensor,
               handle: int) -> Optional[torch.Tensor]:
    """The caller's workspace, or one kept for this stream (calls on one stream do not
    overlap); hold on to it until the launch, as another thread's larger call, or one on
    yet another stream, replaces the kept one.  A captured call needs the caller's own: a later, larger call would
    free the kept one under the graph."""
    if given is not None:
        _same_device(like.device, workspace=given)
        if not given.is_contiguous():
            raise ValueError("workspace must be contiguous")
        return given
    if not nbytes:
        return None
    if torch.cuda.is_current_stream_capturing():
        raise ValueError(f"a captured call needs a workspace of its own (zeroed, {nbytes} bytes)")
    key = (like.get_device(), handle)
    ws = _stream_workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=like.device)
        with _lock:
            # (made on its own stream, so that calls still running there are done
            # before the allocator gives the memory to anyone else)
            _stream_workspaces.pop(key, None)
            while len(_stream_workspaces) >= _KEPT_WORKSPACES:
                del _stream_workspaces[next(iter(_stream_workspaces))]
            _stream_workspaces[key] = ws
    return ws


def _same_device(device: torch.device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


def _check_norm_rope(q, k, v, k_cache, v_cache, slot_mapping, positions, cos_sin, q_weight,
                     k_weight, q_out, fp8):
    """Raises what is wrong with the tensors of _norm_rope_store, by name."""
    NB, bs, Hkv, D = (_fp8_pool_dims if fp8 else _pool_dims)(k_cache, v_cache)
    _need(q, "q", torch.bfloat16, 3, contiguous=False)
    T, Hq = q.shape[0], q.shape[1]
    for name, t, heads in (("q", q, Hq), ("k", k, Hkv), ("v", v, Hkv)):
        _need(t, name, torch.bfloat16, 3, contiguous=False)
        if tuple(t.shape) != (T, heads, D):
            raise ValueError(f"{name} must be [{T}, {heads}, {D}], got {tuple(t.shape)}")
        if T and (t.stride(2) != 1 or (heads > 1 and t.stride(1) != D)):
            raise ValueError(f"{name} must have contiguous rows")
    _need(slot_mapping, "slot_mapping", torch.int32, 1)
    if cos_sin is not None:
        _need(cos_sin, "cos_sin", torch.float32, 2)
        _need(positions, "positions", torch.int32, 1)
    for name, t in (("slot_mapping", slot_mapping),
                    ("positions", positions if cos_sin is not None else None)):
        if t is not None and t.shape[0] != T:
            raise ValueError(f"{name} and q disagree on T")
    for name, t in (("q_weight", q_weight), ("k_weight", k_weight)):
        if t is not None:
            _need(t, name, torch.float32, 1)
            if t.shape[0] != D:
                raise ValueError(f"{name} must be [{D}]")
    if q_out is not None:
        _need(q_out, "q_out", torch.bfloat16, 3)
        if q_out.shape != q.shape:
            raise ValueError("q_out and q differ in shape")
    _same_device(k_cache.device, q=q, k=k, v=v, v_cache=v_cache, slot_mapping=slot_mapping,
                 positions=positions if cos_sin is not None else None, cos_sin=cos_sin,
                 q_weight=q_weight, k_weight=k_weight, q_out=q_out)


def _norm_rope_store(q, k, v, k_cache, v_cache, slot_mapping, positions, cos_sin, q_weight,
                     k_weight, eps, interleaved, q_out, stream, scales):
    lib = _lib or load_library()
    bf16, f32 = torch.bfloat16, torch.float32
    dtype = bf16 if scales is None else torch.uint8
    fine = False
    try:   # every check at once; _check_norm_rope says which one failed
        NB, bs, Hkv, D = pool = k_cache.shape
        T, Hq, _ = shape = q.shape
        kv, row, one = (T, Hkv, D), (D,), (T,)
        at = k_cache.get_device()
        qs, ks, vs = q.stride(), k.stride(), v.stride()
        fine = (
            at >= 0 and shape == (T, Hq, D) and k.shape == kv and v.shape == kv
            and v_cache.shape == pool and slot_mapping.shape == one
            and k_cache.dtype is dtype and v_cache.dtype is dtype
            and q.dtype is bf16 and k.dtype is bf16 and v.dtype is bf16
            and slot_mapping.dtype is torch.int32
            and qs[2] == 1 and ks[2] == 1 and vs[2] == 1
            and (qs[1] == D or Hq == 1) and ((ks[1] == D and vs[1] == D) or Hkv == 1)
            and k_cache.is_contiguous() and v_cache.is_contiguous()
            and slot_mapping.is_contiguous()
            and q.get_device() == at and k.get_device() == at and v.get_device() == at
            and v_cache.get_device() == at and slot_mapping.get_device() == at
            and (cos_sin is None or (
                cos_sin.dtype is f32 and cos_sin.dim() == 2 and cos_sin.is_contiguous()
                and cos_sin.get_device() == at and positions.dtype is torch.int32
                and positions.shape == one and positions.is_contiguous()
                and positions.get_device() == at))
            and (q_weight is None or (q_weight.dtype is f32 and q_weight.shape == row
                                      and q_weight.is_contiguous()
                                      and q_weight.get_device() == at))
            and (k_weight is None or (k_weight.dtype is f32 and k_weight.shape == row
                                      and k_weight.is_contiguous()
                                      and k_weight.get_device() == at))
            and (q_out is None or (q_out.dtype is bf16 and q_out.shape == shape
                                   and q_out.is_contiguous() and q_out.get_device() == at)))
    except (AttributeError, ValueError, TypeError):
        pass
    if not fine:
        _check_norm_rope(q, k, v, k_cache, v_cache, slot_mapping, positions, cos_sin, q_weight,
                         k_weight, q_out, scales is not None)
    if stream is not None or at != _current_device():
        with _Launch(k_cache.device, stream):
            return _norm_rope_store(q, k, v, k_cache, v_cache, slot_mapping, positions, cos_sin,
                                    q_weight, k_weight, eps, interleaved, q_out, None, scales)
    if q_out is None:
        q_out = torch.empty(shape, dtype=bf16, device=q.device)
    places, rotary = (0, 0) if cos_sin is None else cos_sin.shape
    if T < 2:   # a single row's token stride says nothing (torch may give it any value)
        qs, ks, vs = (Hq * D,), (Hkv * D,), (Hkv * D,)
    args = (q_out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), qs[0], ks[0], vs[0],
            k_cache.data_ptr(), v_cache.data_ptr(), slot_mapping.data_ptr(),
            positions.data_ptr() if rotary else None, cos_sin.data_ptr() if rotary else None,
            places, rotary, 1 if interleaved else 0,
            None if q_weight is None else q_weight.data_ptr(),
            None if k_weight is None else k_weight.data_ptr(), float(eps), T, Hq, Hkv, D, bs, NB)
    if scales is None:
        status = lib.kv_cache_store_norm_rope(*args, _current_stream(at))
    else:
        status = lib.kv_cache_store_norm_rope_fp8(*args, float(scales[0]), float(scales[1]),
                                                  _current_stream(at))
    if status != PKV_OK:
        raise PkvError(status, "kv_cache_store_norm_rope" + ("" if scales is None else "_fp8"))
    return q_out


def kv_cache_store_norm_rope(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                             k_cache: torch.Tensor, v_cache: torch.Tensor,
                             slot_mapping: torch.Tensor, positions: Optional[torch.Tensor],
                             cos_sin: Optional[torch.Tensor],
                             q_weight: Optional[torch.Tensor] = None,
                             k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                             interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                             stream=None) -> torch.Tensor:
    """RMS norm of every query and key head, rotation by position, and the store
    of K/V, in one launch.  q bf16 [T, Hq, D], k / v bf16 [T, Hkv, D] (token
    stride free: slices of one packed projection will do); positions int32 [T];
    cos_sin fp32 [max_positions, R]: R/2 cosines, then R/2 sines (None: no
    rotation); q_weight / k_weight fp32 [D] (None: that tensor is not normed).
    Returns the queries, bf16 [T, Hq, D] (q_out; it may be q if q is
    contiguous)."""
    return _norm_rope_store(q, k, v, k_cache, v_cache, slot_mapping, positions, cos_sin, q_weight,
                            k_weight, eps, interleaved, q_out, stream, None)


def kv_cache_store_norm_rope_fp8(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                 k_cache: torch.Tensor, v_cache: torch.Tensor,
                                 slot_mapping: torch.Tensor, positions: Optional[torch.Tensor],
                                 cos_sin: Optional[torch.Tensor], k_scale: float, v_scale: float,
                                 q_weight: Optional[torch.Tensor] = None,
                                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                                 interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                                 stream=None) -> torch.Tensor:
    """kv_cache_store_norm_rope into uint8 E4M3 pools (one scale per tensor)."""
    return _norm_rope_store(q, k, v, k_cache, v_cache, slot_mapping, positions, cos_sin, q_weight,
                            k_weight, eps, interleaved, q_out, stream, (k_scale, v_scale))


def _int32(name: str, value) -> int:
    """`value` as the library's 32-bit int (ctypes would keep its low 32 bits)."""
    n = int(value)
    if not -0x80000000 <= n <= 0x7fffffff:
        raise ValueError(f"{name} = {n} does not fit 32 bits")
    return n


@functools.lru_cache(maxsize=256)
def _scored_workspace_bytes(device_index, B, Hq, Hkv, D, maxblk, bs, window, fp8,
                            num_splits) -> int:
    return int(load_library().paged_decode_scored_workspace_bytes(B, Hq, Hkv, D, maxblk, bs,
                                                                  window, fp8, num_splits))


def paged_decode_scored_workspace_bytes(B: int, Hq: int, Hkv: int, D: int,
                                        max_blocks_per_seq: int, block_size: int = 256,
                                        window: int = 0, num_splits: int = 0,
                                        fp8: bool = False) -> int:
    """Workspace of a scored decode call of these sizes on the current device."""
    sizes = {"B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "max_blocks_per_seq": max_blocks_per_seq,
             "block_size": block_size, "window": window, "fp8": fp8, "num_splits": num_splits}
    return int(load_library().paged_decode_scored_workspace_bytes(
        *(_int32(name, value) for name, value in sizes.items())))


def _check_scored(q, k_cache, v_cache, block_tables, ints, rows, batch, alibi_slopes, first_keys,
                  prefix_lens, out, lse, fp8):
    """Raises what is wrong with the tensors of a scored call, by name."""
    NB, bs, Hkv, D = (_fp8_pool_dims if fp8 else _pool_dims)(k_cache, v_cache)
    _need(q, "q", torch.bfloat16, 3)
    if q.shape[2] != D:
        raise ValueError("q head_dim differs from the cache's")
    _need(block_tables, "block_tables", torch.int32, 2)
    if block_tables.shape[0] != batch:
        raise ValueError(f"block_tables must have {batch} rows")
    for name, (t, n) in ints.items():
        _need(t, name, torch.int32, 1)
        if t.shape[0] != n:
            raise ValueError(f"{name} must be [{n}]")
    for name, t, dtype, n in (("alibi_slopes", alibi_slopes, torch.float32, q.shape[1]),
                              ("first_keys", first_keys, torch.int32, rows),
                              ("prefix_lens", prefix_lens, torch.int32, batch)):
        if t is not None:
            _need(t, name, dtype, 1)
            if t.shape[0] != n:
                raise ValueError(f"{name} must be [{n}]")
    if out is not None:
        _need(out, "out", torch.bfloat16, 3)
        if out.shape != q.shape:
            raise ValueError("out and q differ in shape")
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
        if lse.shape != q.shape[:2]:
            raise ValueError(f"lse must be {tuple(q.shape[:2])}")
    _same_device(q.device, k_cache=k_cache, v_cache=v_cache, block_tables=block_tables,
                 alibi_slopes=alibi_slopes, first_keys=first_keys, prefix_lens=prefix_lens,
                 out=out, lse=lse, **{name: t for name, (t, _) in ints.items()})


def _scored_fine(q, k_cache, v_cache, block_tables, lens, lens2, n_lens, rows, batch, alibi_slopes,
                 first_keys, prefix_lens, out, lse, dtype) -> bool:
    """Whether the tensors of a scored call pass every check (_check_scored says
    which one failed)."""
    i32 = torch.int32
    try:
        shape, pool = q.shape, k_cache.shape
        at = q.get_device()

        def vector(t, kind, n):
            return (t.dtype is kind and t.shape == (n,) and t.is_contiguous()
                    and t.get_device() == at)

        return (
            at >= 0 and len(shape) == 3 and len(pool) == 4 and shape[2] == pool[3]
            and v_cache.shape == pool and k_cache.dtype is dtype and v_cache.dtype is dtype
            and q.dtype is torch.bfloat16 and block_tables.dtype is i32
            and block_tables.dim() == 2 and block_tables.shape[0] == batch
            and q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()
            and block_tables.is_contiguous()
            and k_cache.get_device() == at and v_cache.get_device() == at
            and block_tables.get_device() == at
            and vector(lens, i32, n_lens) and (lens2 is None or vector(lens2, i32, n_lens))
            and (alibi_slopes is None or vector(alibi_slopes, torch.float32, shape[1]))
            and (first_keys is None or vector(first_keys, i32, rows))
            and (prefix_lens is None or vector(prefix_lens, i32, batch))
            and (out is None or (out.dtype is torch.bfloat16 and out.shape == shape
                                 and out.is_contiguous() and out.get_device() == at))
            and (lse is None or (lse.dtype is torch.float32 and lse.shape == shape[:2]
                                 and lse.is_contiguous() and lse.get_device() == at)))
    except (AttributeError, ValueError, TypeError, IndexError):
        return False


def _score_options(softcap, alibi_slopes, window, first_keys, prefix_lens=None) -> ScoreOptions:
    softcap = float(softcap)
    if 0.0 < abs(softcap) < 1e-44:   # 32 bits would hold 0, which is no cap at all
        raise ValueError(f"softcap = {softcap} is too small")
    return ScoreOptions(softcap, window,
                        None if alibi_slopes is None else alibi_slopes.data_ptr(),
                        None if first_keys is None else first_keys.data_ptr(),
                        None if prefix_lens is None else prefix_lens.data_ptr())


def _decode_scored(q, k_cache, v_cache, block_tables, context_lens, scale, scales, softcap,
                   alibi_slopes, window, first_keys, out, lse, workspace, num_splits, want_lse,
                   stream):
    lib = _lib or load_library()
    fp8 = scales is not None
    window, num_splits = _int32("window", window), _int32("num_splits", num_splits)
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    B = q.shape[0] if q.dim() else 0
    if not _scored_fine(q, k_cache, v_cache, block_tables, context_lens, None, B, B, B,
                        alibi_slopes, first_keys, None, out, lse,
                        torch.uint8 if fp8 else torch.bfloat16):
        _check_scored(q, k_cache, v_cache, block_tables, {"context_lens": (context_lens, B)}, B, B,
                      alibi_slopes, first_keys, None, out, lse, fp8)
    at = q.get_device()
    if stream is not None or at != _current_device():
        with _Launch(q.device, stream):
            return _decode_scored(q, k_cache, v_cache, block_tables, context_lens, scale, scales,
                                  softcap, alibi_slopes, window, first_keys, out, lse, workspace,
                                  num_splits, want_lse, None)
    Hq = q.shape[1]
    NB, bs, Hkv, D = k_cache.shape
    maxblk = block_tables.shape[1]
    handle = _current_stream(at)
    need = _scored_workspace_bytes(at, B, Hq, Hkv, D, maxblk, bs, window, int(fp8), num_splits)
    ws = _workspace(workspace, need, q, handle) if need or workspace is not None else None
    at_ws, ws_bytes = (0, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    args = (out.data_ptr(), None if lse is None else lse.data_ptr(), q.data_ptr(),
            k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), maxblk,
            context_lens.data_ptr(), B, Hq, Hkv, D, bs, NB, float(scale))
    options = _score_options(softcap, alibi_slopes, window, first_keys)
    if fp8:
        status = lib.paged_decode_attention_scored_fp8(*args, float(scales[0]), float(scales[1]),
                                                       options, at_ws, ws_bytes, num_splits, handle)
    else:
        status = lib.paged_decode_attention_scored(*args, options, at_ws, ws_bytes, num_splits,
                                                   handle)
    if status != PKV_OK:
        raise PkvError(status, "paged_decode_attention_scored" + ("_fp8" if fp8 else ""))
    return out, lse


def paged_decode_attention_scored(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                  block_tables: torch.Tensor, context_lens: torch.Tensor,
                                  scale: float, softcap: float = 0.0,
                                  alibi_slopes: Optional[torch.Tensor] = None, window: int = 0,
                                  first_keys: Optional[torch.Tensor] = None,
                                  out: Optional[torch.Tensor] = None,
                                  lse: Optional[torch.Tensor] = None,
                                  workspace: Optional[torch.Tensor] = None, num_splits: int = 0,
                                  want_lse: bool = True, stream=None
                                  ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """paged_decode_attention with scores capped by softcap * tanh(s / softcap),
    biased by -alibi_slopes[h] * distance (fp32 [Hq]), and restricted to the last
    `window` keys and to keys from first_keys[b] on (int32 [B]).  Returns (out
    bf16 [B, Hq, D], lse fp32 [B, Hq] or None).  Without a given workspace one is
    kept per stream; a captured call needs its own."""
    return _decode_scored(q, k_cache, v_cache, block_tables, context_lens, scale, None, softcap,
                          alibi_slopes, window, first_keys, out, lse, workspace, num_splits,
                          want_lse, stream)


def paged_decode_attention_scored_fp8(q: torch.Tensor, k_cache: torch.Tensor,
                                      v_cache: torch.Tensor, block_tables: torch.Tensor,
                                      context_lens: torch.Tensor, scale: float, k_scale: float,
                                      v_scale: float, softcap: float = 0.0,
                                      alibi_slopes: Optional[torch.Tensor] = None,
                                      window: int = 0, first_keys: Optional[torch.Tensor] = None,
                                      out: Optional[torch.Tensor] = None,
                                      lse: Optional[torch.Tensor] = None,
                                      workspace: Optional[torch.Tensor] = None,
                                      num_splits: int = 0, want_lse: bool = True, stream=None
                                      ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """paged_decode_attention_scored over uint8 E4M3 pools."""
    return _decode_scored(q, k_cache, v_cache, block_tables, context_lens, scale,
                          (k_scale, v_scale), softcap, alibi_slopes, window, first_keys, out, lse,
                          workspace, num_splits, want_lse, stream)


def paged_prefill_attention_scored(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                   block_tables: torch.Tensor, cu_seqlens_q: torch.Tensor,
                                   cu_seqlens_k: torch.Tensor, max_seqlen_q: int,
                                   max_seqlen_k: int, scale: float, softcap: float = 0.0,
                                   alibi_slopes: Optional[torch.Tensor] = None, window: int = 0,
                                   first_keys: Optional[torch.Tensor] = None,
                                   prefix_lens: Optional[torch.Tensor] = None,
                                   out: Optional[torch.Tensor] = None,
                                   lse: Optional[torch.Tensor] = None, want_lse: bool = True,
                                   stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """paged_prefill_attention with the options of paged_decode_attention_scored
    (first_keys: int32, one per query row) and prefix_lens (int32 [B]): rows inside
    the first prefix_lens[b] tokens of sequence b see up to the last of them.  Values
    may be as large as 2^32.  Returns (out bf16 [sum Lq, Hq, D], lse fp32
    [sum Lq, Hq] or None)."""
    lib = _lib or load_library()
    window = _int32("window", window)
    max_seqlen_q = _int32("max_seqlen_q", max_seqlen_q)
    max_seqlen_k = _int32("max_seqlen_k", max_seqlen_k)
    for name, t in (("q", q), ("block_tables", block_tables)):
        if not isinstance(t, torch.Tensor) or not t.dim():
            raise TypeError(f"{name} must be a torch.Tensor with rows")
    Nq = q.shape[0]
    B = block_tables.shape[0]
    if not _scored_fine(q, k_cache, v_cache, block_tables, cu_seqlens_q, cu_seqlens_k, B + 1, Nq, B,
                        alibi_slopes, first_keys, prefix_lens, out, lse, torch.bfloat16):
        _check_scored(q, k_cache, v_cache, block_tables,
                      {"cu_seqlens_q": (cu_seqlens_q, B + 1),
                       "cu_seqlens_k": (cu_seqlens_k, B + 1)},
                      Nq, B, alibi_slopes, first_keys, prefix_lens, out, lse, False)
    at = q.get_device()
    if stream is not None or at != _current_device():
        with _Launch(q.device, stream):
            return paged_prefill_attention_scored(
                q, k_cache, v_cache, block_tables, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                max_seqlen_k, scale, softcap, alibi_slopes, window, first_keys, prefix_lens, out,
                lse, want_lse)
    Hq = q.shape[1]
    NB, bs, Hkv, D = k_cache.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((Nq, Hq), dtype=torch.float32, device=q.device)
    status = lib.paged_prefill_attention_scored(
        out.data_ptr(), None if lse is None else lse.data_ptr(), q.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), block_tables.shape[1],
        cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), B, Nq, max_seqlen_q,
        max_seqlen_k, Hq, Hkv, D, bs, NB, float(scale),
        _score_options(softcap, alibi_slopes, window, first_keys, prefix_lens),
        _current_stream(at))
    if status != PKV_OK:
        raise PkvError(status, "paged_prefill_attention_scored")
    return out, lse


def testing_set_wait_fault(wait_limit_ns: int, withhold_tile: int = -1) -> None:
    """For tests only: lower the kernels' wait limit and make the copy
    producers withhold one tile (see pkv_testing_set_wait_fault in pkv.h);
    testing_set_wait_fault(0, -1) turns it off."""
    _check(load_library().pkv_testing_set_wait_fault(int(wait_limit_ns), int(withhold_tile)),
           "pkv_testing_set_wait_fault")


def get_device_error(stream=None) -> int:
    """Synchronise the stream and read-and-clear the device error word."""
    return int(load_library().pkv_get_device_error(_stream(stream)))
