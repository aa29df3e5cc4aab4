"""Thin Python binding of libffd.so (ctypes): argument marshalling only.

Every entry point has the name of its C counterpart in include/ffd.h and forwards torch tensors
as raw device pointers. Nothing here computes any step of the method; a missing or unloadable
library raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import NamedTuple

import torch

from . import _build

_lock = threading.Lock()
_lib = None

FFD_OK = 0
FFD_ERR_CUDA = 4
STATUS_NAMES = {0: "FFD_OK", 1: "FFD_ERR_INVALID_ARG", 2: "FFD_ERR_UNSUPPORTED",
                3: "FFD_ERR_WORKSPACE", 4: "FFD_ERR_CUDA", 5: "FFD_ERR_BOUNDS",
                6: "FFD_ERR_RANGE", 7: "FFD_ERR_TIMEOUT"}
HEAD_DIM = 128
PAGE = 64
SCHEDULE_FUSED = 0        # FFD_SCHEDULE_FUSED
SCHEDULE_SCAN_REFINE = 1  # FFD_SCHEDULE_SCAN_REFINE


class FFDError(RuntimeError):
    def __init__(self, status: int, where: str, cuda_error: int = 0):
        self.status = status
        self.cuda_error = cuda_error
        extra = f" (cudaError_t {cuda_error})" if cuda_error else ""
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}{extra}")


class CacheDesc(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32)]


class DecodeParams(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32), ("sink_tokens", ctypes.c_int32),
                ("local_tokens", ctypes.c_int32), ("delta", ctypes.c_float),
                ("sm_scale", ctypes.c_float), ("num_splits", ctypes.c_int32),
                ("wait_limit_us", ctypes.c_int32), ("schedule", ctypes.c_int32)]


class Kv4Params(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("max_q_len", ctypes.c_int32), ("total_q", ctypes.c_int32),
                ("window", ctypes.c_int32), ("num_splits", ctypes.c_int32),
                ("q_stride", ctypes.c_int64), ("sm_scale", ctypes.c_float),
                ("wait_limit_us", ctypes.c_int32)]


class RopeParams(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("total_tokens", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("rot_scale", ctypes.c_float),
                ("q_stride", ctypes.c_int64), ("q_out_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64)]


class TreeParams(ctypes.Structure):
    _fields_ = Kv4Params._fields_


def make_params(batch, num_q_heads, num_kv_heads, num_pages, max_blocks_per_seq, *, sink=64,
                local=1024, delta=5.0, sm_scale=None, num_splits=0,
                wait_limit_us=0, schedule=0) -> DecodeParams:
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    return DecodeParams(batch, num_q_heads, num_kv_heads, HEAD_DIM, PAGE, num_pages,
                        max_blocks_per_seq, sink, local, delta, sm_scale, num_splits,
                        wait_limit_us, schedule)


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """Load libffd.so (built in-tree by ``__graft_entry__.build()``)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_build.LIB):
                raise RuntimeError(f"{_build.LIB} is missing: build it with "
                                   "`python -c 'import __graft_entry__ as g; g.build()'`")
            L = ctypes.CDLL(_build.LIB)
            P = ctypes.c_void_p
            st = ctypes.c_int
            L.ffd_status_string.argtypes = [st]
            L.ffd_status_string.restype = ctypes.c_char_p
            L.ffd_version.argtypes = []
            L.ffd_version.restype = ctypes.c_int32
            L.ffd_last_cuda_error.argtypes = []
            L.ffd_last_cuda_error.restype = ctypes.c_int32
            L.ffd_suggest_schedule.argtypes = [ctypes.c_int64, ctypes.c_int64]
            L.ffd_suggest_schedule.restype = ctypes.c_int32
            L.ffd_quantize_keys.argtypes = [ctypes.POINTER(CacheDesc), P, P, P, P,
                                            ctypes.c_int32, P, P]
            L.ffd_quantize_keys.restype = st
            L.ffd_append_kv.argtypes = [ctypes.POINTER(CacheDesc), ctypes.c_int32,
                                        ctypes.c_int32] + [P] * 10
            L.ffd_append_kv.restype = st
            L.ffd_decode_workspace_size.argtypes = [ctypes.POINTER(DecodeParams)]
            L.ffd_decode_workspace_size.restype = ctypes.c_size_t
            L.ffd_dense_workspace_size.argtypes = [ctypes.POINTER(DecodeParams)]
            L.ffd_dense_workspace_size.restype = ctypes.c_size_t
            L.ffd_decode_attention.argtypes = [ctypes.POINTER(DecodeParams)] + [P] * 10 + \
                [ctypes.c_size_t, P]
            L.ffd_decode_attention.restype = st
            L.ffd_dense_decode.argtypes = [ctypes.POINTER(DecodeParams)] + [P] * 7 + \
                [ctypes.c_size_t, P]
            L.ffd_dense_decode.restype = st
            L.ffd_decode_attention_static.argtypes = [ctypes.POINTER(DecodeParams)] + \
                [P] * 11
            L.ffd_decode_attention_static.restype = st
            L.ffd_select_workspace_size.argtypes = [ctypes.POINTER(DecodeParams)]
            L.ffd_select_workspace_size.restype = ctypes.c_size_t
            L.ffd_select_blocks.argtypes = [ctypes.POINTER(DecodeParams), ctypes.c_int32,
                                            ctypes.c_float] + [P] * 6 + [ctypes.c_size_t, P]
            L.ffd_select_blocks.restype = st
            L.ffd_decode_attention_masked.argtypes = [ctypes.POINTER(DecodeParams)] + \
                [P] * 11 + [ctypes.c_size_t, P]
            L.ffd_decode_attention_masked.restype = st
            L.ffd_art_workspace_size.argtypes = [ctypes.POINTER(DecodeParams)]
            L.ffd_art_workspace_size.restype = ctypes.c_size_t
            L.ffd_art_attention.argtypes = [ctypes.POINTER(DecodeParams), ctypes.c_float,
                                            ctypes.c_float, ctypes.c_int32] + [P] * 10 + \
                [ctypes.c_size_t, P]
            L.ffd_art_attention.restype = st
            i32, i64 = ctypes.c_int32, ctypes.c_int64
            L.ffd_kv4_write.argtypes = [ctypes.POINTER(CacheDesc), i32, i32, i32, i32, P, i64, P,
                                        i64] + [P] * 7
            L.ffd_kv4_write.restype = st
            L.ffd_kv4_read.argtypes = [ctypes.POINTER(CacheDesc), i32, i32, i32, i32] + [P] * 6 + \
                [i64, P, i64, P, P]
            L.ffd_kv4_read.restype = st
            L.ffd_kv4_workspace_size.argtypes = [ctypes.POINTER(Kv4Params)]
            L.ffd_kv4_workspace_size.restype = ctypes.c_size_t
            L.ffd_kv4_attention.argtypes = [ctypes.POINTER(Kv4Params)] + [P] * 10 + \
                [ctypes.c_size_t, P]
            L.ffd_kv4_attention.restype = st
            L.ffd_rope_append.argtypes = [ctypes.POINTER(RopeParams)] + [P] * 15
            L.ffd_rope_append.restype = st
            L.ffd_tree_workspace_size.argtypes = [ctypes.POINTER(TreeParams)]
            L.ffd_tree_workspace_size.restype = ctypes.c_size_t
            L.ffd_tree_attention.argtypes = [ctypes.POINTER(TreeParams)] + [P] * 11 + \
                [ctypes.c_size_t, P]
            L.ffd_tree_attention.restype = st
            L.ffd_tree_commit.argtypes = [ctypes.POINTER(CacheDesc), i32, i32, i32] + [P] * 16
            L.ffd_tree_commit.restype = st
            L.ffd_set_profile_events.argtypes = [P, P]
            L.ffd_set_profile_events.restype = st
            L.ffd_get_error.argtypes = [P, P]
            L.ffd_get_error.restype = st
            _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check(status: int, where: str):
    if status != FFD_OK:
        raise FFDError(status, where,
                       ffd_last_cuda_error() if status == FFD_ERR_CUDA else 0)


THUMB_RECORD_BYTES = 3072
RESID_RECORD_BYTES = 8704


class QuantizedCache(NamedTuple):
    """The stored key cache, one record pair per (page, KV head), byte layouts in include/ffd.h:
    thumb u8 [P, Hkv, 3072] (2-bit codes, thumbnail scales, zeros); resid u8 [P, Hkv, 8704]
    (int8 residual codes in the kernel's chunk order, residual scales)."""
    thumb: torch.Tensor
    resid: torch.Tensor


def alloc_quantized_cache(num_pages: int, num_kv_heads: int, device="cuda") -> QuantizedCache:
    shp = (num_pages, num_kv_heads)
    return QuantizedCache(
        torch.empty(shp + (THUMB_RECORD_BYTES,), dtype=torch.uint8, device=device),
        torch.empty(shp + (RESID_RECORD_BYTES,), dtype=torch.uint8, device=device))


def ffd_status_string(status: int) -> str:
    return lib().ffd_status_string(status).decode()


def ffd_version() -> int:
    return int(lib().ffd_version())


def ffd_suggest_schedule(total_blocks: int, kept_blocks: int) -> int:
    """SCHEDULE_FUSED or SCHEDULE_SCAN_REFINE for a step like the previous one (host only)."""
    return int(lib().ffd_suggest_schedule(int(total_blocks), int(kept_blocks)))


def ffd_last_cuda_error() -> int:
    """The cudaError_t behind this thread's latest FFD_ERR_CUDA (0 if none)."""
    return int(lib().ffd_last_cuda_error())


def ffd_quantize_keys(k: torch.Tensor, cache: QuantizedCache, *, page_ids=None,
                      error_word=None, stream=None) -> None:
    """Quantise bf16 keys k [P,Hkv,64,128] into ``cache`` (all pages, or ``page_ids``)."""
    desc = CacheDesc(k.shape[0], k.shape[1], k.shape[3], k.shape[2])
    n_ids = 0 if page_ids is None else int(page_ids.numel())
    _check(lib().ffd_quantize_keys(ctypes.byref(desc), _ptr(k), *map(_ptr, cache),
                                   _ptr(page_ids), n_ids, _ptr(error_word), _stream(stream)),
           "ffd_quantize_keys")


def ffd_append_kv(k_new, v_new, positions, block_table, cache: QuantizedCache, v_cache, *,
                  k_cache=None, error_word=None, stream=None) -> None:
    """Append one token per sequence: k_new, v_new bf16 [B,Hkv,128] go to row p % 64 of page
    block_table[b, p // 64], p = positions[b] (negative: nothing for that sequence)."""
    P, Hkv = v_cache.shape[0], v_cache.shape[1]
    desc = CacheDesc(P, Hkv, v_cache.shape[3], v_cache.shape[2])
    _check(lib().ffd_append_kv(ctypes.byref(desc), k_new.shape[0], block_table.shape[1],
                               _ptr(k_new), _ptr(v_new), _ptr(positions), _ptr(block_table),
                               *map(_ptr, cache), _ptr(v_cache), _ptr(k_cache),
                               _ptr(error_word), _stream(stream)), "ffd_append_kv")


def ffd_decode_workspace_size(params: DecodeParams) -> int:
    return int(lib().ffd_decode_workspace_size(ctypes.byref(params)))


def ffd_dense_workspace_size(params: DecodeParams) -> int:
    return int(lib().ffd_dense_workspace_size(ctypes.byref(params)))


def alloc_workspace(params: DecodeParams, *, dense=False, device="cuda") -> torch.Tensor:
    """Zero-filled workspace of the size the library asks for (torch allocates it)."""
    n = ffd_dense_workspace_size(params) if dense else ffd_decode_workspace_size(params)
    if n == 0:
        raise FFDError(1, "workspace size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def ffd_decode_attention(params: DecodeParams, q, cache: QuantizedCache, v, seq_lens,
                         block_table, out, workspace, *, keep_mask=None, m_tilde=None,
                         stream=None) -> None:
    _check(lib().ffd_decode_attention(
        ctypes.byref(params), _ptr(q), *map(_ptr, cache), _ptr(v), _ptr(seq_lens),
        _ptr(block_table), _ptr(out), _ptr(keep_mask), _ptr(m_tilde), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)), "ffd_decode_attention")


def ffd_decode_attention_static(params: DecodeParams, q, cache: QuantizedCache, v, seq_lens,
                                block_table, out, *, keep_mask=None, m_tilde=None,
                                error_word=None, stream=None) -> None:
    """ffd_decode_attention without a workspace, for callers that cannot allocate device memory:
    the library's own 4 MiB static device scratch is used instead (calls that overlap on the GPU
    race on it; the first call on a device should precede any stream capture)."""
    _check(lib().ffd_decode_attention_static(
        ctypes.byref(params), _ptr(q), *map(_ptr, cache), _ptr(v), _ptr(seq_lens),
        _ptr(block_table), _ptr(out), _ptr(keep_mask), _ptr(m_tilde), _ptr(error_word),
        _stream(stream)), "ffd_decode_attention_static")


SELECT_TOPK = 1
SELECT_TOPP = 2


def ffd_select_workspace_size(params: DecodeParams) -> int:
    return int(lib().ffd_select_workspace_size(ctypes.byref(params)))


def alloc_select_workspace(params: DecodeParams, device="cuda") -> torch.Tensor:
    n = ffd_select_workspace_size(params)
    if n == 0:
        raise FFDError(1, "select workspace size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def ffd_select_blocks(params: DecodeParams, selector: int, budget: float, q, cache: QuantizedCache,
                      seq_lens, block_table, keep_mask, workspace, *, stream=None) -> None:
    """Top-k (selector 1, budget = k) or Top-p (selector 2, budget = p) block mask."""
    _check(lib().ffd_select_blocks(
        ctypes.byref(params), selector, budget, _ptr(q), _ptr(cache.thumb), _ptr(seq_lens),
        _ptr(block_table), _ptr(keep_mask), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)), "ffd_select_blocks")


def ffd_decode_attention_masked(params: DecodeParams, q, cache: QuantizedCache, v, seq_lens,
                                block_table, keep_in, out, workspace, *, keep_mask=None,
                                m_tilde=None, stream=None) -> None:
    """Exact attention over the blocks a given mask selects (the decode workspace)."""
    _check(lib().ffd_decode_attention_masked(
        ctypes.byref(params), _ptr(q), *map(_ptr, cache), _ptr(v), _ptr(seq_lens),
        _ptr(block_table), _ptr(keep_in), _ptr(out), _ptr(keep_mask), _ptr(m_tilde),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)),
        "ffd_decode_attention_masked")


def ffd_art_workspace_size(params: DecodeParams) -> int:
    return int(lib().ffd_art_workspace_size(ctypes.byref(params)))


def alloc_art_workspace(params: DecodeParams, device="cuda") -> torch.Tensor:
    n = ffd_art_workspace_size(params)
    if n == 0:
        raise FFDError(1, "ART workspace size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def ffd_art_attention(params: DecodeParams, tau: float, phi: float, patience: int, q,
                      cache: QuantizedCache, v, seq_lens, block_table, out, workspace, *,
                      keep_in=None, blocks_used=None, stream=None) -> None:
    """Attention with run-time termination (ART) over block 0 and the blocks of ``keep_in`` (all
    blocks when None), most recent first; ``blocks_used`` [B, Hkv] int32 receives the count."""
    _check(lib().ffd_art_attention(
        ctypes.byref(params), tau, phi, patience, _ptr(q), *map(_ptr, cache), _ptr(v),
        _ptr(seq_lens), _ptr(block_table), _ptr(keep_in), _ptr(out), _ptr(blocks_used),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)),
        "ffd_art_attention")


def ffd_dense_decode(params: DecodeParams, q, k, v, seq_lens, block_table, out, workspace, *,
                     stream=None) -> None:
    _check(lib().ffd_dense_decode(
        ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(seq_lens), _ptr(block_table),
        _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)), "ffd_dense_decode")

# ---- the 4-bit cache ----------------------------------------------------------------------------
KV4_RECORD_BYTES = 5120
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}  # FFD_DTYPE_BF16, FFD_DTYPE_F16


class Kv4Cache(NamedTuple):
    """Keys and values in 4 bits, one record per (page, KV head) each (layout in include/ffd.h):
    k4, v4 u8 [P, Hkv, 5120]."""
    k4: torch.Tensor
    v4: torch.Tensor


def alloc_kv4_cache(num_pages: int, num_kv_heads: int, device="cuda") -> Kv4Cache:
    shp = (num_pages, num_kv_heads, KV4_RECORD_BYTES)
    return Kv4Cache(torch.empty(shp, dtype=torch.uint8, device=device),
                    torch.empty(shp, dtype=torch.uint8, device=device))


# The three calls below check their tensors in one flat expression each: a decode step takes about as
# long on the host as on the GPU, and every function call and attribute that is read counts.
# (torch._C's two lookups are there in CUDA builds alone, which importing this does not ask for)
_C = torch._C
_I32, _U8, _F32 = torch.int32, torch.uint8, torch.float32
_descs = {}  # (P, Hkv) -> a reference to its CacheDesc


def _refuse(where: str, what: str):
    raise FFDError(1, f"{where}: {what}")


def _desc(P: int, Hkv: int):
    ref = _descs.get((P, Hkv))
    if ref is None:
        ref = _descs[(P, Hkv)] = ctypes.byref(CacheDesc(P, Hkv, HEAD_DIM, PAGE))
    return ref


def _stream_of(stream, dev: int) -> int:
    if stream is None:
        return _C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _row_stride(x, rows: int, heads: int, dtype):
    """Elements between the rows of x [rows, heads, 128], or None when it is not such rows."""
    if x.dtype != dtype or x.shape != (rows, heads, HEAD_DIM):
        return None
    t, h, c = x.stride()
    if rows == 0:
        return heads * HEAD_DIM
    if c != 1 or (h != HEAD_DIM and heads > 1):
        return None
    return t if rows > 1 else heads * HEAD_DIM


def _kv4_rows(where, cache, positions, block_table, k, v, cu_tokens, error_word):
    """Checks of a write or a read: (device, P, Hkv, B, table width, rows, dtype, strides of k, v)."""
    k4, v4 = cache
    one = v if k is None else k
    if one is None:
        _refuse(where, "no rows")
    dev = k4.get_device()
    if not (dev >= 0 and v4.get_device() == dev and positions.get_device() == dev
            and block_table.get_device() == dev and (k is None or k.get_device() == dev)
            and (v is None or v.get_device() == dev)
            and (cu_tokens is None or cu_tokens.get_device() == dev)
            and (error_word is None or error_word.get_device() == dev)):
        _refuse(where, "tensors on different devices, or not on a GPU")
    shape, table = k4.shape, block_table.shape
    if not (k4.dtype == _U8 and v4.dtype == _U8 and len(shape) == 3 and shape[2] == KV4_RECORD_BYTES
            and v4.shape == shape and k4.is_contiguous() and v4.is_contiguous()):
        _refuse(where, "the cache")
    if len(table) != 2 or not (
            block_table.dtype == _I32 and positions.dtype == _I32
            and positions.shape == table[:1] and block_table.is_contiguous()
            and positions.is_contiguous()
            and (cu_tokens is None or (cu_tokens.dtype == _I32 and cu_tokens.is_contiguous()
                                       and cu_tokens.shape == (table[0] + 1,)))):
        _refuse(where, "int32 positions [B], cu_tokens [B + 1], block_table [B, width]")
    if error_word is not None and error_word.nbytes < 4:
        _refuse(where, "an error word of 4 bytes")
    P, Hkv, _ = shape
    T, dtype = one.shape[0], one.dtype
    ks = 0 if k is None else _row_stride(k, T, Hkv, dtype)
    vs = 0 if v is None else _row_stride(v, T, Hkv, dtype)
    if ks is None or vs is None or dtype not in _DTYPES:
        _refuse(where, "rows of bf16 or fp16 [T, Hkv, 128]")
    return dev, P, Hkv, table[0], table[1], T, dtype, ks, vs


def _addr(t):
    return None if t is None else t.data_ptr()


def ffd_kv4_write(k_new, v_new, positions, block_table, cache: Kv4Cache, *, cu_tokens=None,
                  error_word=None, stream=None) -> None:
    """Quantise rows k_new, v_new [T, Hkv, 128] (bf16 or fp16; rows may lie inside wider ones) into
    the 4-bit cache. Sequence b's rows are cu_tokens[b] .. cu_tokens[b+1]-1 (T / B each when None)
    and go to tokens positions[b], positions[b]+1, ... (negative: nothing for that sequence)."""
    where = "ffd_kv4_write"
    if k_new is None or v_new is None:
        _refuse(where, "no rows")
    dev, P, Hkv, B, width, T, dtype, ks, vs = _kv4_rows(where, cache, positions, block_table, k_new,
                                                        v_new, cu_tokens, error_word)
    if _C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return ffd_kv4_write(k_new, v_new, positions, block_table, cache, cu_tokens=cu_tokens,
                                 error_word=error_word, stream=stream)
    status = (_lib or lib()).ffd_kv4_write(
        _desc(P, Hkv), _DTYPES[dtype], B, width, T, k_new.data_ptr(), ks, v_new.data_ptr(), vs,
        _addr(cu_tokens), positions.data_ptr(), block_table.data_ptr(), cache[0].data_ptr(),
        cache[1].data_ptr(), _addr(error_word), _stream_of(stream, dev))
    if status != FFD_OK:
        _check(status, where)


def ffd_kv4_read(cache: Kv4Cache, positions, block_table, k_out, v_out, *, cu_tokens=None,
                 error_word=None, stream=None) -> None:
    """The values the 4-bit cache holds, as rows k_out, v_out [T, Hkv, 128] (bf16 or fp16; either
    may be None). Rows and tokens are matched as in ffd_kv4_write."""
    where = "ffd_kv4_read"
    dev, P, Hkv, B, width, T, dtype, ks, vs = _kv4_rows(where, cache, positions, block_table, k_out,
                                                        v_out, cu_tokens, error_word)
    if _C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return ffd_kv4_read(cache, positions, block_table, k_out, v_out, cu_tokens=cu_tokens,
                                error_word=error_word, stream=stream)
    status = (_lib or lib()).ffd_kv4_read(
        _desc(P, Hkv), _DTYPES[dtype], B, width, T, _addr(cu_tokens), positions.data_ptr(),
        block_table.data_ptr(), cache[0].data_ptr(), cache[1].data_ptr(), _addr(k_out), ks,
        _addr(v_out), vs, _addr(error_word), _stream_of(stream, dev))
    if status != FFD_OK:
        _check(status, where)


def make_kv4_params(batch, num_q_heads, num_kv_heads, num_pages, max_blocks_per_seq, *,
                    max_q_len=1, total_q=None, dtype=torch.bfloat16, window=0, sm_scale=None,
                    num_splits=0, q_stride=0, wait_limit_us=0) -> Kv4Params:
    """total_q None: every sequence has max_q_len query tokens."""
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    if total_q is None:
        total_q = batch * max_q_len
    return Kv4Params(batch, num_q_heads, num_kv_heads, HEAD_DIM, PAGE, num_pages,
                     max_blocks_per_seq, _DTYPES[dtype], max_q_len, total_q, window, num_splits,
                     q_stride, sm_scale, wait_limit_us)


def ffd_kv4_workspace_size(params: Kv4Params) -> int:
    return int(lib().ffd_kv4_workspace_size(ctypes.byref(params)))


def alloc_kv4_workspace(params: Kv4Params, device="cuda") -> torch.Tensor:
    n = ffd_kv4_workspace_size(params)
    if n == 0:
        raise FFDError(1, "4-bit attention workspace size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def ffd_kv4_attention(params: Kv4Params, q, cache: Kv4Cache, seq_lens, block_table, out, workspace,
                      *, cu_q=None, keep_in=None, lse=None, stream=None) -> None:
    """Attention of each sequence's newest tokens over its 4-bit cache: q [total_q, Hq, 128], rows
    params.q_stride elements apart, out [total_q, Hq, 128], lse fp32 [total_q, Hq] or None."""
    where = "ffd_kv4_attention"
    k4, v4 = cache
    dev = q.get_device()
    if not (dev >= 0 and k4.get_device() == dev and v4.get_device() == dev
            and seq_lens.get_device() == dev and block_table.get_device() == dev
            and out.get_device() == dev and workspace.get_device() == dev
            and (cu_q is None or cu_q.get_device() == dev)
            and (keep_in is None or keep_in.get_device() == dev)
            and (lse is None or lse.get_device() == dev)):
        _refuse(where, "tensors on different devices, or not on a GPU")
    B, Hq, Hkv, T = params.batch, params.num_q_heads, params.num_kv_heads, params.total_q
    width, dtype, row = params.max_blocks_per_seq, q.dtype, Hq * HEAD_DIM
    shape = (params.num_pages, Hkv, KV4_RECORD_BYTES)
    if not (k4.dtype == _U8 and v4.dtype == _U8 and k4.shape == shape and v4.shape == shape
            and k4.is_contiguous() and v4.is_contiguous()):
        _refuse(where, "the cache")
    shape = (T, Hq, HEAD_DIM)
    if not (q.shape == shape and out.shape == shape and out.dtype == dtype and out.is_contiguous()
            and _DTYPES.get(dtype) == params.dtype):
        _refuse(where, "q and out of params.dtype [total_q, Hq, 128]")
    stride = q.stride()
    if (stride[2] != 1 or (stride[1] != HEAD_DIM and Hq > 1)
            or (T > 1 and stride[0] != (params.q_stride or row))):
        _refuse(where, "q's rows, params.q_stride elements apart")
    if not (block_table.dtype == _I32 and block_table.shape == (B, width)
            and block_table.is_contiguous() and seq_lens.dtype == _I32 and seq_lens.shape == (B,)
            and seq_lens.is_contiguous()
            and (cu_q is None or (cu_q.dtype == _I32 and cu_q.shape == (B + 1,)
                                  and cu_q.is_contiguous()))):
        _refuse(where, "int32 seq_lens [B], cu_q [B + 1], block_table [B, max_blocks_per_seq]")
    if keep_in is not None and not (keep_in.dtype == _U8 and keep_in.shape == (B, Hkv, width)
                                    and keep_in.is_contiguous()):
        _refuse(where, "keep_in u8 [B, Hkv, max_blocks_per_seq]")
    if lse is not None and not (lse.dtype == _F32 and lse.shape == (T, Hq) and lse.is_contiguous()):
        _refuse(where, "lse fp32 [total_q, Hq]")
    if not workspace.is_contiguous():
        _refuse(where, "the workspace")
    if _C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return ffd_kv4_attention(params, q, cache, seq_lens, block_table, out, workspace,
                                     cu_q=cu_q, keep_in=keep_in, lse=lse, stream=stream)
    status = (_lib or lib()).ffd_kv4_attention(
        ctypes.byref(params), q.data_ptr(), k4.data_ptr(), v4.data_ptr(), seq_lens.data_ptr(),
        _addr(cu_q), block_table.data_ptr(), _addr(keep_in), out.data_ptr(), _addr(lse),
        workspace.data_ptr(), workspace.nbytes, _stream_of(stream, dev))
    if status != FFD_OK:
        _check(status, where)


# ---- speculative decoding over the 16-bit cache -------------------------------------------------
TREE_MAX_NODES = 256
_I64 = torch.int64
_rope_shapes = {}  # shape of an append -> a reference to its RopeParams


def _records(quantized, P, Hkv, dev):
    thumb, resid = quantized
    return (thumb.dtype == _U8 and resid.dtype == _U8 and thumb.shape == (P, Hkv, THUMB_RECORD_BYTES)
            and resid.shape == (P, Hkv, RESID_RECORD_BYTES) and thumb.is_contiguous()
            and resid.is_contiguous() and thumb.get_device() == dev and resid.get_device() == dev)


# (checks are written out flat here too, see above)
def ffd_rope_append(q, k_new, v_new, inv_freq, positions, block_table, q_out, k_cache, v_cache, *,
                    cu_tokens=None, rope_positions=None, interleaved=False, rot_scale=1.0,
                    quantized=None, error_word=None, stream=None) -> None:
    """Rotate q [T, Hq, 128] into q_out (both None: no queries; the same tensor: in place) and
    k_new [T, Hkv, 128] into the cache, and append v_new: k_cache, v_cache [P, Hkv, 64, 128] of the rows'
    dtype (k_cache may be None where ``quantized``, a QuantizedCache, is given). The first
    2 * inv_freq.numel() channels are rotated (inv_freq fp32 or None), by rope_positions int32 [T] or
    the tokens' own indices. Rows and tokens are matched as in ffd_kv4_write."""
    where = "ffd_rope_append"
    if (k_new is None or v_new is None or v_cache is None or (q is None) != (q_out is None)
            or (k_cache is None and quantized is None)):
        _refuse(where, "rows, or a cache for them, missing")
    dev, dtype, cache, new, table = (v_cache.get_device(), k_new.dtype, v_cache.shape, k_new.shape,
                                     block_table.shape)
    if not (dev >= 0 and k_new.get_device() == dev and v_new.get_device() == dev
            and positions.get_device() == dev and block_table.get_device() == dev
            and (k_cache is None or k_cache.get_device() == dev)
            and (q is None or (q.get_device() == dev and q_out.get_device() == dev))
            and (inv_freq is None or inv_freq.get_device() == dev)
            and (rope_positions is None or rope_positions.get_device() == dev)
            and (cu_tokens is None or cu_tokens.get_device() == dev)
            and (error_word is None or error_word.get_device() == dev)):
        _refuse(where, "tensors on different devices, or not on a GPU")
    code = _DTYPES.get(dtype)
    if not (code is not None and len(cache) == 4 and cache[2] == PAGE and cache[3] == HEAD_DIM
            and v_cache.dtype is dtype and v_cache.is_contiguous()
            and (k_cache is None or (k_cache.dtype is dtype and k_cache.shape == cache
                                     and k_cache.is_contiguous()))):
        _refuse(where, "k_cache and v_cache [P, Hkv, 64, 128] of the rows' dtype, bf16 or fp16")
    P, Hkv = cache[0], cache[1]
    if quantized is not None and not _records(quantized, P, Hkv, dev):
        _refuse(where, "the quantised cache")
    if len(table) != 2 or not (
            block_table.dtype is _I32 and block_table.is_contiguous() and positions.dtype is _I32
            and positions.shape == table[:1] and positions.is_contiguous()
            and (cu_tokens is None or (cu_tokens.dtype is _I32 and cu_tokens.is_contiguous()
                                       and cu_tokens.shape == (table[0] + 1,)))):
        _refuse(where, "int32 positions [B], cu_tokens [B + 1], block_table [B, width]")
    if not (len(new) == 3 and new[1] == Hkv and new[2] == HEAD_DIM and v_new.dtype is dtype
            and v_new.shape == new):
        _refuse(where, "rows of one dtype: k_new, v_new [T, Hkv, 128]")
    T, rot = new[0], 0
    if rope_positions is not None and not (rope_positions.dtype is _I32 and rope_positions.shape == (T,)
                                           and rope_positions.is_contiguous()):
        _refuse(where, "int32 rope_positions [T]")
    if inv_freq is not None:
        if not (inv_freq.dtype is _F32 and inv_freq.dim() == 1 and inv_freq.is_contiguous()):
            _refuse(where, "inv_freq fp32 [rotated channels / 2]")
        rot = 2 * inv_freq.numel()
    if error_word is not None and error_word.nbytes < 4:
        _refuse(where, "an error word of 4 bytes")
    # elements between rows, which may lie inside wider ones
    ks, a, b = k_new.stride()
    vs, c, d = v_new.stride()
    row, fine = Hkv * HEAD_DIM, b == 1 and d == 1 and (Hkv == 1 or a == c == HEAD_DIM)
    if T <= 1:
        ks, vs, fine = row, row, fine or T == 0
    Hq = qs = qos = 0
    if q is not None and fine:
        shape = q.shape
        fine = (len(shape) == 3 and shape[0] == T and shape[2] == HEAD_DIM and q.dtype is dtype
                and q_out.dtype is dtype and q_out.shape == shape)
        if fine:
            Hq = shape[1]
            qs, a, b = q.stride()
            qos, c, d = q_out.stride()
            fine = b == 1 and d == 1 and (Hq == 1 or a == c == HEAD_DIM)
            if T <= 1:
                qs, qos, fine = Hq * HEAD_DIM, Hq * HEAD_DIM, fine or T == 0
    if not fine:
        _refuse(where, "rows of one dtype: q, q_out [T, Hq, 128], k_new, v_new [T, Hkv, 128]")
    if _C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return ffd_rope_append(q, k_new, v_new, inv_freq, positions, block_table, q_out, k_cache,
                                   v_cache, cu_tokens=cu_tokens, rope_positions=rope_positions,
                                   interleaved=interleaved, rot_scale=rot_scale, quantized=quantized,
                                   error_word=error_word, stream=stream)
    shape = (table[0], Hq, Hkv, HEAD_DIM, PAGE, P, table[1], code, T, rot, 1 if interleaved else 0,
             rot_scale, qs, qos, ks, vs)
    ref = _rope_shapes.get(shape)
    if ref is None:
        if len(_rope_shapes) >= 1024:  # ragged batches come in many sizes
            _rope_shapes.clear()
        ref = _rope_shapes[shape] = ctypes.byref(RopeParams(*shape))
    thumb, resid = (None, None) if quantized is None else (t.data_ptr() for t in quantized)
    status = (_lib or lib()).ffd_rope_append(
        ref, None if q is None else q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
        None if inv_freq is None else inv_freq.data_ptr(),
        None if rope_positions is None else rope_positions.data_ptr(),
        None if cu_tokens is None else cu_tokens.data_ptr(), positions.data_ptr(),
        block_table.data_ptr(), None if q is None else q_out.data_ptr(),
        None if k_cache is None else k_cache.data_ptr(), v_cache.data_ptr(), thumb, resid,
        None if error_word is None else error_word.data_ptr(),
        _C._cuda_getCurrentRawStream(dev) if stream is None else _stream_of(stream, dev))
    if status != FFD_OK:
        _check(status, where)


def make_tree_params(batch, num_q_heads, num_kv_heads, num_pages, max_blocks_per_seq, *,
                     max_q_len=1, total_q=None, dtype=torch.bfloat16, window=0, sm_scale=None,
                     num_splits=0, q_stride=0, wait_limit_us=0) -> TreeParams:
    """total_q None: every sequence has max_q_len nodes."""
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    if total_q is None:
        total_q = batch * max_q_len
    return TreeParams(batch, num_q_heads, num_kv_heads, HEAD_DIM, PAGE, num_pages,
                      max_blocks_per_seq, _DTYPES[dtype], max_q_len, total_q, window, num_splits,
                      q_stride, sm_scale, wait_limit_us)


def ffd_tree_workspace_size(params: TreeParams) -> int:
    return int(lib().ffd_tree_workspace_size(ctypes.byref(params)))


def alloc_tree_workspace(params: TreeParams, device="cuda") -> torch.Tensor:
    n = ffd_tree_workspace_size(params)
    if n == 0:
        raise FFDError(1, "tree attention workspace size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def ffd_tree_attention(params: TreeParams, q, k, v, seq_lens, block_table, out, workspace, *,
                       parents=None, cu_q=None, keep_in=None, lse=None, stream=None) -> None:
    """Attention of each sequence's newest tokens, a tree of drafted tokens (parents int32 [total_q],
    -1 or an earlier node of the sequence; None: a chain), over k, v [P, Hkv, 64, 128]:
    q [total_q, Hq, 128], rows params.q_stride elements apart, out [total_q, Hq, 128], lse fp32
    [total_q, Hq] or None."""
    where = "ffd_tree_attention"
    dev = q.get_device()
    if not (dev >= 0 and k.get_device() == dev and v.get_device() == dev
            and seq_lens.get_device() == dev and block_table.get_device() == dev
            and out.get_device() == dev and workspace.get_device() == dev
            and (parents is None or parents.get_device() == dev)
            and (cu_q is None or cu_q.get_device() == dev)
            and (keep_in is None or keep_in.get_device() == dev)
            and (lse is None or lse.get_device() == dev)):
        _refuse(where, "tensors on different devices, or not on a GPU")
    B, Hq, Hkv, T = params.batch, params.num_q_heads, params.num_kv_heads, params.total_q
    width, dtype, row = params.max_blocks_per_seq, q.dtype, Hq * HEAD_DIM
    shape = (params.num_pages, Hkv, PAGE, HEAD_DIM)
    if not (k.dtype == dtype and v.dtype == dtype and k.shape == shape and v.shape == shape
            and k.is_contiguous() and v.is_contiguous()):
        _refuse(where, "k and v [num_pages, Hkv, 64, 128] of q's dtype")
    shape = (T, Hq, HEAD_DIM)
    if not (q.shape == shape and out.shape == shape and out.dtype == dtype and out.is_contiguous()
            and _DTYPES.get(dtype) == params.dtype):
        _refuse(where, "q and out of params.dtype [total_q, Hq, 128]")
    stride = q.stride()
    if (stride[2] != 1 or (stride[1] != HEAD_DIM and Hq > 1)
            or (T > 1 and stride[0] != (params.q_stride or row))):
        _refuse(where, "q's rows, params.q_stride elements apart")
    if not (block_table.dtype == _I32 and block_table.shape == (B, width)
            and block_table.is_contiguous() and seq_lens.dtype == _I32 and seq_lens.shape == (B,)
            and seq_lens.is_contiguous()
            and (parents is None or (parents.dtype == _I32 and parents.shape == (T,)
                                     and parents.is_contiguous()))
            and (cu_q is None or (cu_q.dtype == _I32 and cu_q.shape == (B + 1,)
                                  and cu_q.is_contiguous()))):
        _refuse(where, "int32 seq_lens [B], parents [total_q], cu_q [B + 1], block_table [B, "
                       "max_blocks_per_seq]")
    if keep_in is not None and not (keep_in.dtype == _U8 and keep_in.shape == (B, Hkv, width)
                                    and keep_in.is_contiguous()):
        _refuse(where, "keep_in u8 [B, Hkv, max_blocks_per_seq]")
    if lse is not None and not (lse.dtype == _F32 and lse.shape == (T, Hq) and lse.is_contiguous()):
        _refuse(where, "lse fp32 [total_q, Hq]")
    if not workspace.is_contiguous():
        _refuse(where, "the workspace")
    if _C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return ffd_tree_attention(params, q, k, v, seq_lens, block_table, out, workspace,
                                      parents=parents, cu_q=cu_q, keep_in=keep_in, lse=lse,
                                      stream=stream)
    status = (_lib or lib()).ffd_tree_attention(
        ctypes.byref(params), q.data_ptr(), k.data_ptr(), v.data_ptr(), seq_lens.data_ptr(),
        _addr(cu_q), _addr(parents), block_table.data_ptr(), _addr(keep_in), out.data_ptr(),
        _addr(lse), workspace.data_ptr(), workspace.nbytes, _stream_of(stream, dev))
    if status != FFD_OK:
        _check(status, where)


def ffd_tree_commit(draft, target, seq_lens, block_table, k_cache, v_cache, path, accepted, next_token,
                    new_lens, *, parents=None, cu_nodes=None, quantized=None, error_word=None,
                    stream=None) -> None:
    """Accept the drafted tokens that the model confirms (draft int64 [T], target int64 [T]: the
    model's token behind each node) and move their rows to the sequences' ends. k_cache (or None)
    and v_cache [P, Hkv, 64, 128], ``quantized`` a QuantizedCache or None; outputs path int32 [T],
    accepted and new_lens int32 [B], next_token int64 [B]."""
    where = "ffd_tree_commit"
    dev, cache, table, nodes = v_cache.get_device(), v_cache.shape, block_table.shape, draft.shape
    if not (dev >= 0 and draft.get_device() == dev and target.get_device() == dev
            and seq_lens.get_device() == dev and block_table.get_device() == dev
            and path.get_device() == dev and accepted.get_device() == dev
            and next_token.get_device() == dev and new_lens.get_device() == dev
            and (k_cache is None or k_cache.get_device() == dev)
            and (parents is None or parents.get_device() == dev)
            and (cu_nodes is None or cu_nodes.get_device() == dev)
            and (error_word is None or error_word.get_device() == dev)):
        _refuse(where, "tensors on different devices, or not on a GPU")
    if not (len(cache) == 4 and cache[2] == PAGE and cache[3] == HEAD_DIM and v_cache.dtype in _DTYPES
            and v_cache.is_contiguous()
            and (k_cache is None or (k_cache.dtype is v_cache.dtype and k_cache.shape == cache
                                     and k_cache.is_contiguous()))):
        _refuse(where, "k_cache and v_cache [P, Hkv, 64, 128], bf16 or fp16")
    if quantized is not None and not _records(quantized, cache[0], cache[1], dev):
        _refuse(where, "the quantised cache")
    if len(table) != 2 or not (
            block_table.dtype is _I32 and block_table.is_contiguous()
            and seq_lens.dtype is _I32 and seq_lens.shape == table[:1] and seq_lens.is_contiguous()
            and accepted.dtype is _I32 and accepted.shape == table[:1] and accepted.is_contiguous()
            and new_lens.dtype is _I32 and new_lens.shape == table[:1] and new_lens.is_contiguous()
            and next_token.dtype is _I64 and next_token.shape == table[:1] and next_token.is_contiguous()
            and (cu_nodes is None or (cu_nodes.dtype is _I32 and cu_nodes.is_contiguous()
                                      and cu_nodes.shape == (table[0] + 1,)))):
        _refuse(where, "int32 seq_lens, accepted, new_lens [B], cu_nodes [B + 1], block_table [B, width],"
                       " int64 next_token [B]")
    if len(nodes) != 1 or not (
            draft.dtype is _I64 and draft.is_contiguous() and target.dtype is _I64
            and target.shape == nodes and target.is_contiguous() and path.dtype is _I32
            and path.shape == nodes and path.is_contiguous()
            and (parents is None or (parents.dtype is _I32 and parents.shape == nodes
                                     and parents.is_contiguous()))):
        _refuse(where, "int64 draft, target [T], int32 path, parents [T]")
    if error_word is not None and error_word.nbytes < 4:
        _refuse(where, "an error word of 4 bytes")
    if _C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return ffd_tree_commit(draft, target, seq_lens, block_table, k_cache, v_cache, path,
                                   accepted, next_token, new_lens, parents=parents, cu_nodes=cu_nodes,
                                   quantized=quantized, error_word=error_word, stream=stream)
    thumb, resid = (None, None) if quantized is None else (t.data_ptr() for t in quantized)
    ref = _descs.get(cache[:2])
    status = (_lib or lib()).ffd_tree_commit(
        _desc(cache[0], cache[1]) if ref is None else ref, table[0], table[1], nodes[0],
        draft.data_ptr(), target.data_ptr(), None if parents is None else parents.data_ptr(),
        None if cu_nodes is None else cu_nodes.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(),
        None if k_cache is None else k_cache.data_ptr(), v_cache.data_ptr(), thumb, resid,
        path.data_ptr(), accepted.data_ptr(), next_token.data_ptr(), new_lens.data_ptr(),
        None if error_word is None else error_word.data_ptr(),
        _C._cuda_getCurrentRawStream(dev) if stream is None else _stream_of(stream, dev))
    if status != FFD_OK:
        _check(status, where)


def ffd_get_error(error_word, *, stream=None) -> int:
    """Synchronise, read and clear a device error word; returns the status code."""
    return int(lib().ffd_get_error(_ptr(error_word), _stream(stream)))


def ffd_set_profile_events(start=None, stop=None) -> None:
    """Record ``start`` / ``stop`` (torch.cuda.Event, created) around the main kernel of the
    following decode calls; ``None, None`` turns it off."""
    def raw(ev):
        if ev is None:
            return None
        return ctypes.c_void_p(ev.cuda_event)
    _check(lib().ffd_set_profile_events(raw(start), raw(stop)), "ffd_set_profile_events")
