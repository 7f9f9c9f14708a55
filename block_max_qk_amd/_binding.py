"""ctypes binding of libmsa_index_score.so (argument marshalling only).

Every step of the operator runs in the HIP library; this module only turns
torch tensors into the C ABI's plain descriptors and pointers, passes torch's
current HIP stream, and turns a non-zero status into an exception.  If the
library is missing the call raises: there is no fallback implementation.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import operator
import os
import struct
import threading
from typing import NamedTuple, Optional, Sequence

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmsa_index_score.so")

# msa_dtype_t / msa_layout_t / msa_status_t of include/msa_index_score.h
DTYPE_CODE = {
    torch.float16: 0,
    torch.bfloat16: 1,
    torch.int8: 2,
    torch.float8_e4m3fn: 3,
    torch.float8_e5m2: 4,
    torch.uint8: 5,          # MXFP4: E2M1 pairs, with E8M0 group scales alongside
}
LAYOUT_CODE = {"TND": 0, "BBND": 1, "BNBD": 2}
STATUS_NAMES = ["MSA_OK", "MSA_ERR_NULL", "MSA_ERR_LAYOUT", "MSA_ERR_DTYPE", "MSA_ERR_SHAPE",
                "MSA_ERR_STRIDE", "MSA_ERR_SCALE", "MSA_ERR_ATTR", "MSA_ERR_HIP",
                "MSA_ERR_WORKSPACE"]
EXPORTED = ("msa_index_score", "msa_index_score_family", "msa_index_score_ex",
            "msa_index_score_mxfp4", "msa_index_score_mxfp4_family",
            "msa_index_score_out_width", "msa_status_str",
            "msa_index_score_kernel_family", "msa_block_topk", "msa_cache_append",
            "msa_attention", "msa_block_attention", "msa_attention_workspace",
            "msa_attention_tile_rows", "msa_step_tables", "msa_cache_append_axes",
            "msa_attention_ex", "msa_attention_ex_workspace")
LOCAL_MODE_CODE = {"request": 0, "query": 1}


class MsaTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


class MsaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES[status] if 0 <= status < len(STATUS_NAMES) else status}: "
                         f"{message}")
        self.status = status


class MsaLayoutError(MsaError, ValueError):
    pass


_lock = threading.Lock()
_lib = None


def load_library(path: Optional[str] = None):
    """Load the HIP library (built in-tree by ``block_max_qk_amd.build``)."""
    global _lib
    with _lock:
        if path is None and _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"HIP library {p} is not built; run "
                               "`python -m block_max_qk_amd.build` (hipcc, gfx950)")
        lib = ctypes.CDLL(p)
        ptr = ctypes.c_void_p
        i32 = ctypes.c_int32
        # query, key, start_loc, block_table, max_blocks, scale, cu_seqlens_q,
        # kv_len, batch, block_size, layout, sparse_mode, init_blocks,
        # local_blocks, out, out_width, stream
        args = [ctypes.POINTER(MsaTensor), ctypes.POINTER(MsaTensor), ptr, ptr, ctypes.c_int64,
                ptr, ptr, ptr, i32, i32, i32, i32, i32, i32, ptr, ctypes.c_int64, ptr]
        lib.msa_index_score.argtypes = args
        lib.msa_index_score.restype = ctypes.c_int
        lib.msa_index_score_family.argtypes = args + [i32]
        lib.msa_index_score_family.restype = ctypes.c_int
        # local_mode after local_blocks, family last
        lib.msa_index_score_ex.argtypes = args[:14] + [i32] + args[14:] + [i32]
        lib.msa_index_score_ex.restype = ctypes.c_int
        lib.msa_index_score_mxfp4.argtypes = [
            ctypes.POINTER(MsaTensor), ptr, ctypes.POINTER(MsaTensor), ptr, ptr, ptr,
            ctypes.c_int64, ptr, ptr, i32, i32, i32, i32, i32, i32, i32, ptr, ctypes.c_int64,
            ptr]
        lib.msa_index_score_mxfp4.restype = ctypes.c_int
        lib.msa_index_score_mxfp4_family.argtypes = (lib.msa_index_score_mxfp4.argtypes +
                                                     [ctypes.c_int32])
        lib.msa_index_score_mxfp4_family.restype = ctypes.c_int
        lib.msa_index_score_out_width.argtypes = [ctypes.c_int64]
        lib.msa_index_score_out_width.restype = ctypes.c_int64
        lib.msa_status_str.argtypes = [ctypes.c_int32]
        lib.msa_status_str.restype = ctypes.c_char_p
        lib.msa_index_score_kernel_family.argtypes = [ctypes.c_int64, ctypes.c_int32,
                                                      ctypes.c_int32, ctypes.c_int32]
        lib.msa_index_score_kernel_family.restype = ctypes.c_int32
        lib.msa_block_topk.argtypes = [ptr, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                       ctypes.c_int64, ctypes.c_int32, ptr, ptr]
        lib.msa_block_topk.restype = ctypes.c_int
        i64 = ctypes.c_int64
        # items, num_items, cos, sin, positions, rotary_dim, interleaved,
        # block_table, max_blocks, cu_seqlens_q, kv_len, batch, block_size, stream
        lib.msa_cache_append.argtypes = [ptr, i32, ptr, ptr, i64, i32, i32, ptr, i64, ptr, ptr,
                                         i32, i32, ptr]
        lib.msa_cache_append.restype = ctypes.c_int
        # axis_positions, axes, pair_axes (host bytes) after interleaved
        args = lib.msa_cache_append.argtypes
        lib.msa_cache_append_axes.argtypes = [*args[:7], ptr, i32, ctypes.c_char_p, *args[7:]]
        lib.msa_cache_append_axes.restype = ctypes.c_int
        # block_table, max_blocks, cu_seqlens_q, kv_len, batch, block_size,
        # layout, sparse_mode, softmax_scale, out, lse, workspace,
        # workspace_bytes, stream
        tail = [ptr, i64, ptr, ptr, i32, i32, i32, i32, ctypes.c_float, ptr, ptr, ptr, i64, ptr]
        three = [ptr] * 3                # descriptors, as packed bytes or byref()
        lib.msa_attention.argtypes = three + tail
        lib.msa_attention.restype = ctypes.c_int
        # softcap, slopes, visible after softmax_scale
        lib.msa_attention_ex.argtypes = three + tail[:9] + [ctypes.c_float, ptr, ptr] + tail[9:]
        lib.msa_attention_ex.restype = ctypes.c_int
        lib.msa_attention_ex_workspace.argtypes = [i64, i32, i32, i32, i64]
        lib.msa_attention_ex_workspace.restype = i64
        lib.msa_block_attention.argtypes = three + [ptr, i32] + tail
        lib.msa_block_attention.restype = ctypes.c_int
        lib.msa_attention_workspace.argtypes = [i64, i32, i32, i32, i64, i32]
        lib.msa_attention_workspace.restype = i64
        lib.msa_attention_tile_rows.argtypes = [i64, i32, i32, i32, i64, i32]
        lib.msa_attention_tile_rows.restype = i32
        # new_tokens, ctx_len, rows, batch, pool, pool_rows, pool_blocks,
        # free_pages, free_size, free_count, free_out, max_blocks, T, block_size,
        # cu_seqlens_q, kv_len, start_loc, block_table, positions, slots,
        # cu_pages, stream
        lib.msa_step_tables.argtypes = [ptr, ptr, ptr, i32, ptr, i64, i64, ptr, i64, ptr, ptr, i64,
                                        i64, i32, ptr, ptr, ptr, ptr, ptr, ptr, ptr, ptr]
        lib.msa_step_tables.restype = ctypes.c_int
        if path is None:
            _lib = lib
        return lib


def describe(t: torch.Tensor, dtype_code: Optional[int] = None) -> MsaTensor:
    """Descriptor of a tensor: data pointer, element type, shape, strides."""
    d = MsaTensor()
    d.data = t.data_ptr() if t.numel() else (t.data_ptr() or None)
    d.dtype = DTYPE_CODE.get(t.dtype, -1) if dtype_code is None else dtype_code
    d.ndim = t.dim()
    for i in range(min(t.dim(), 4)):
        d.shape[i] = t.shape[i]
        d.stride[i] = t.stride(i)
    return d


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _layout_code(layout) -> int:
    if isinstance(layout, str):
        return LAYOUT_CODE.get(layout.upper(), -1)
    return int(layout)


def msa_index_score_out_width(max_blocks: int) -> int:
    return int(load_library().msa_index_score_out_width(int(max_blocks)))


def msa_status_str(status: int) -> str:
    return load_library().msa_status_str(int(status)).decode()


def msa_index_score_kernel_family(T: int, batch: int, Hq: int, Hkv: int) -> int:
    return int(load_library().msa_index_score_kernel_family(int(T), int(batch), int(Hq),
                                                            int(Hkv)))


BLOCK_SIZE = 128   # tokens per logical block (guide to msa_index_score, section 四)
MASK_SHAPE = (2048, 2048)   # the compressed causal template of sparse_mode 3


def _stream_handle(stream, dev):
    if stream is None:
        return torch.cuda.current_stream(dev).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return stream


def _local_mode_code(local_mode) -> int:
    return LOCAL_MODE_CODE.get(local_mode, -1) if isinstance(local_mode, str) else int(local_mode)


def _check_batch(query, out, start_loc, block_table, cu_seqlens_q, kv_len, max_blocks,
                 local_mode) -> int:
    """Sizes the C ABI takes on trust (it sees plain pointers): the request
    count B from kv_len, and the tensors whose extents follow from it and from
    the query.  Returns B."""
    if kv_len.dim() != 1:
        raise ValueError("kv_len must be 1-D [B] (per-request lengths)")
    B = int(kv_len.numel())
    if cu_seqlens_q.dim() != 1 or cu_seqlens_q.numel() != B + 1:
        raise ValueError(f"cu_seqlens_q must be [B+1] = [{B + 1}], got "
                         f"{tuple(cu_seqlens_q.shape)}")
    if start_loc is None:
        if _local_mode_code(local_mode) != 1 and B > 0:
            raise ValueError("start_loc is required unless local_mode is 'query'")
    elif start_loc.dim() != 1 or start_loc.numel() != B:
        raise ValueError(f"start_loc must be [B] = [{B}], got {tuple(start_loc.shape)}")
    if block_table is not None:
        if (block_table.dim() != 2 or block_table.shape[0] < B or
                block_table.shape[1] != int(max_blocks)):
            raise ValueError(f"block_table must be [>= {B}, max_blocks = {int(max_blocks)}], "
                             f"got {tuple(block_table.shape)}")
    if query.dim() == 3 and (out.shape[0] != query.shape[1] or out.shape[1] != query.shape[0]):
        raise ValueError(f"out must be [Hq, T, W] = [{query.shape[1]}, {query.shape[0]}, W], "
                         f"got {tuple(out.shape)}")
    return B


def _key_rows(key: torch.Tensor, layout: int):
    """(rows, Hkv) of a key tensor: token rows of one KV head across the cache
    (NP * 128 paged, T2 packed) and the KV head count, or None if the shape
    does not fit the layout (the C ABI then reports it)."""
    if layout == 0 and key.dim() == 3:
        return key.shape[0], key.shape[1]
    if layout == 1 and key.dim() == 3:
        return key.shape[0] * key.shape[1], 1
    if layout == 1 and key.dim() == 4:
        return key.shape[0] * key.shape[1], key.shape[2]
    if layout == 2 and key.dim() == 4:
        return key.shape[0] * key.shape[2], key.shape[1]
    return None


def _raise_status(st: int):
    if st != 0:
        cls = MsaLayoutError if st == 2 else MsaError
        raise cls(st, msa_status_str(st))


def msa_index_score(query: torch.Tensor, key: torch.Tensor, start_loc: torch.Tensor,
                    block_table: Optional[torch.Tensor], scale: Optional[torch.Tensor],
                    cu_seqlens_q: torch.Tensor, kv_len: torch.Tensor, layout,
                    sparse_mode: int, init_blocks: int, local_blocks: int, out: torch.Tensor,
                    max_blocks: int, stream=None, family: int = -1,
                    local_mode=0, block_size: int = BLOCK_SIZE) -> torch.Tensor:
    """Call the C ABI on device tensors; ``out`` ([Hq, T, W] float32) is filled
    asynchronously on ``stream`` (default: torch's current stream).
    ``kv_len`` holds per-request lengths [B] for every layout.
    ``local_mode`` 0/"request" ends the local window at start_loc, 1/"query"
    at each token's own block (start_loc may then be None)."""
    lib = load_library()
    dev = out.device
    for name, t in (("query", query), ("key", key), ("start_loc", start_loc),
                    ("cu_seqlens_q", cu_seqlens_q), ("kv_len", kv_len),
                    ("block_table", block_table), ("scale", scale)):
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, out on {dev}")
    for name, t in (("start_loc", start_loc), ("cu_seqlens_q", cu_seqlens_q),
                    ("kv_len", kv_len), ("block_table", block_table)):
        if t is not None and (t.dtype != torch.int32 or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous int32 tensor")
    if scale is not None and (scale.dtype != torch.float32 or not scale.is_contiguous()):
        raise ValueError("scale must be a contiguous float32 tensor")
    if out.dtype != torch.float32 or not out.is_contiguous() or out.dim() != 3:
        raise ValueError("out must be a contiguous float32 [Hq, T, W] tensor")
    B = _check_batch(query, out, start_loc, block_table, cu_seqlens_q, kv_len, max_blocks,
                     local_mode)
    lay = _layout_code(layout)
    kr = _key_rows(key, lay)
    if scale is not None and kr is not None and scale.numel() != kr[0] * kr[1]:
        # paged [NP, Hkv, 128], packed [T2, Hkv]: one float per key row and head
        raise ValueError(f"scale must hold {kr[0] * kr[1]} floats (one per key token and KV "
                         f"head), got {scale.numel()}")
    stream = _stream_handle(stream, dev)
    qd, kd = describe(query), describe(key)
    args = (ctypes.byref(qd), ctypes.byref(kd), _ptr(start_loc), _ptr(block_table),
            int(max_blocks), _ptr(scale), _ptr(cu_seqlens_q), _ptr(kv_len), B,
            int(block_size), lay, int(sparse_mode), int(init_blocks), int(local_blocks),
            _ptr(out), int(out.shape[2]), ctypes.c_void_p(stream))
    lm = _local_mode_code(local_mode)
    if lm != 0:
        st = lib.msa_index_score_ex(*args[:14], lm, *args[14:], int(family))
    elif family == -1:
        st = lib.msa_index_score(*args)
    else:
        st = lib.msa_index_score_family(*args, int(family))
    _raise_status(st)
    return out


def msa_index_score_mxfp4(query: torch.Tensor, query_scale: torch.Tensor, key: torch.Tensor,
                          key_scale: torch.Tensor, start_loc: Optional[torch.Tensor],
                          block_table: Optional[torch.Tensor], cu_seqlens_q: torch.Tensor,
                          kv_len: torch.Tensor, layout, sparse_mode: int, init_blocks: int,
                          local_blocks: int, out: torch.Tensor, max_blocks: int, stream=None,
                          local_mode=0, family: int = -1,
                          block_size: int = BLOCK_SIZE) -> torch.Tensor:
    """The MXFP4 entry: ``query`` [T, Hq, 64] and ``key`` (layout-shaped, last
    axis 64) uint8 hold E2M1 pairs; ``query_scale`` [T, Hq, 4] and
    ``key_scale`` (the key's layout with a last axis of 4) uint8 hold E8M0.
    ``family`` -1 picks the kernel family from the sizes, 0/1 force the
    decode/prefill tiles."""
    lib = load_library()
    dev = out.device
    for name, t in (("query", query), ("query_scale", query_scale), ("key", key),
                    ("key_scale", key_scale), ("start_loc", start_loc),
                    ("cu_seqlens_q", cu_seqlens_q), ("kv_len", kv_len),
                    ("block_table", block_table)):
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, out on {dev}")
    for name, t in (("query", query), ("key", key), ("query_scale", query_scale),
                    ("key_scale", key_scale)):
        if t.dtype != torch.uint8:
            raise ValueError(f"{name} must be uint8 (MXFP4 values / E8M0 scales)")
    for name, t in (("start_loc", start_loc), ("cu_seqlens_q", cu_seqlens_q),
                    ("kv_len", kv_len), ("block_table", block_table)):
        if t is not None and (t.dtype != torch.int32 or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous int32 tensor")
    for name, t in (("query_scale", query_scale), ("key_scale", key_scale)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if out.dtype != torch.float32 or not out.is_contiguous() or out.dim() != 3:
        raise ValueError("out must be a contiguous float32 [Hq, T, W] tensor")
    B = _check_batch(query, out, start_loc, block_table, cu_seqlens_q, kv_len, max_blocks,
                     local_mode)
    lay = _layout_code(layout)
    # one E8M0 byte per 32 elements: 4 per 64-byte row
    if query.dim() == 3 and query_scale.numel() != query.shape[0] * query.shape[1] * 4:
        raise ValueError("query_scale must be [T, Hq, 4]")
    kr = _key_rows(key, lay)
    if kr is not None and key_scale.numel() != kr[0] * kr[1] * 4:
        raise ValueError("key_scale must hold 4 bytes per key token and KV head (the key's "
                         "layout with a last axis of 4)")
    stream = _stream_handle(stream, dev)
    qd, kd = describe(query), describe(key)
    st = lib.msa_index_score_mxfp4_family(
        ctypes.byref(qd), _ptr(query_scale), ctypes.byref(kd), _ptr(key_scale),
        _ptr(start_loc), _ptr(block_table), int(max_blocks), _ptr(cu_seqlens_q),
        _ptr(kv_len), B, int(block_size), lay, int(sparse_mode), int(init_blocks),
        int(local_blocks), _local_mode_code(local_mode), _ptr(out), int(out.shape[2]),
        ctypes.c_void_p(stream), int(family))
    _raise_status(st)
    return out


def index_score(query: torch.Tensor, key: torch.Tensor, start_loc: torch.Tensor, *,
                block_table: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                atten_mask: Optional[torch.Tensor] = None,
                actual_seq_qlen: Optional[torch.Tensor] = None,
                actual_seq_klen: Optional[torch.Tensor] = None, layout_key: str = "BBND",
                sparse_mode: int = 3, init_blocks: int = 0, local_blocks: int = 1,
                max_blocks: Optional[int] = None, stream=None, family: int = -1,
                local_mode=0) -> torch.Tensor:
    """The guide's keyword interface (sections 三 and 四): allocate
    ``[Hq, T, RoundUp(MB, 16)]`` float32 and fill it.

    * ``layout_key`` is upper-cased; anything but TND/BBND/BNBD is a ValueError.
    * ``atten_mask``: with ``sparse_mode`` 3 an int8 ``[2048, 2048]`` tensor
      is required, with 0 none may be passed.  It is only checked: the
      right-down causal window is computed from the lengths, the mask
      template is never read.
    * ``actual_seq_qlen``: the ``[B+1]`` query prefix sum.
    * ``actual_seq_klen``: paged layouts take the ``[B]`` per-request lengths,
      TND the ``[B+1]`` prefix sum of the packed key, which is differenced
      into lengths here.
    * MB is ``block_table.shape[1]`` for paged keys; for packed keys pass
      ``max_blocks`` or it is the largest ``ceil(length / 128)``, read from a
      host copy of the lengths (a device synchronisation), ``ceil(T2/128)``
      when the batch is empty.
    """
    lay = layout_key.upper() if isinstance(layout_key, str) else layout_key
    if isinstance(lay, str) and lay not in LAYOUT_CODE:
        raise ValueError(f"layout_key must be one of TND/BBND/BNBD, got {layout_key!r}")
    if int(sparse_mode) == 3:
        if atten_mask is None:
            raise ValueError("sparse_mode 3 needs the [2048, 2048] int8 atten_mask")
        if tuple(atten_mask.shape) != MASK_SHAPE or atten_mask.dtype != torch.int8:
            raise ValueError(f"atten_mask must be int8 {list(MASK_SHAPE)}, got "
                             f"{atten_mask.dtype} {list(atten_mask.shape)}")
    elif atten_mask is not None:
        raise ValueError(f"atten_mask must not be passed with sparse_mode {sparse_mode}")
    if actual_seq_qlen is None or actual_seq_klen is None:
        raise ValueError("actual_seq_qlen and actual_seq_klen are required")
    packed = (lay == "TND") if isinstance(lay, str) else int(lay) == 0
    kv_len = actual_seq_klen
    if packed:
        if actual_seq_klen.dim() != 1 or actual_seq_klen.numel() < 1:
            raise ValueError("TND actual_seq_klen must be the [B+1] key prefix sum")
        kv_len = (actual_seq_klen[1:] - actual_seq_klen[:-1]).to(torch.int32).contiguous()
    if max_blocks is None:
        if block_table is not None:
            max_blocks = int(block_table.shape[1])
        else:
            kv = kv_len.to("cpu", torch.int64)
            max_blocks = (int(((kv + 127) // 128).max()) if kv.numel()
                          else (int(key.shape[0]) + 127) // 128)
    W = msa_index_score_out_width(max_blocks)
    out = torch.empty((query.shape[1], query.shape[0], W), dtype=torch.float32,
                      device=query.device)
    return msa_index_score(query, key, start_loc, block_table, scale, actual_seq_qlen, kv_len,
                           lay, sparse_mode, init_blocks, local_blocks, out, max_blocks,
                           stream=stream, family=family, local_mode=local_mode)


def msa_block_topk(scores: torch.Tensor, num_valid: int, k: int, out: torch.Tensor,
                   stream=None) -> torch.Tensor:
    """Call the C ABI: ``out`` ([T, Hq, k] int32) receives, for every row of
    ``scores`` ([Hq, T, W] float32 on the same device), the k best blocks
    below ``num_valid`` in ascending block order with a -1 tail;
    asynchronous on ``stream`` (default: torch's current stream)."""
    lib = load_library()
    if scores.dtype != torch.float32 or not scores.is_contiguous() or scores.dim() != 3:
        raise ValueError("scores must be a contiguous float32 [Hq, T, W] tensor")
    Hq, T, W = scores.shape
    if out.dtype != torch.int32 or not out.is_contiguous() or tuple(out.shape) != (T, Hq, k):
        raise ValueError(f"out must be a contiguous int32 [{T}, {Hq}, {k}] tensor")
    if out.device != scores.device:
        raise ValueError(f"scores are on {scores.device}, out on {out.device}")
    if stream is None:
        stream = torch.cuda.current_stream(scores.device).cuda_stream
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    st = lib.msa_block_topk(_ptr(scores), Hq, T, W, int(num_valid), int(k), _ptr(out),
                            ctypes.c_void_p(stream))
    if st != 0:
        raise MsaError(st, msa_status_str(st))
    return out


def block_topk(scores: torch.Tensor, num_valid: Optional[int] = None, k: int = 16,
               stream=None) -> torch.Tensor:
    """Allocate ``[T, Hq, k]`` int32 and fill it with the top-k selection of
    the score rows (``num_valid`` defaults to the row width)."""
    Hq, T, W = scores.shape
    out = torch.empty((T, Hq, k), dtype=torch.int32, device=scores.device)
    return msa_block_topk(scores, W if num_valid is None else num_valid, k, out, stream=stream)


# ---------------------------------------------------------------------------
# around the index branch: the cache append and the attention
# ---------------------------------------------------------------------------

ROWS = 3   # MSA_LAYOUT_ROWS: one row per new token, not a cache
APPEND_MAX_ITEMS = 8


class CacheItem(NamedTuple):
    """One tensor of a ``msa_cache_append`` call: ``src`` [T, H, 128] f16/bf16
    rows, rotated if ``rotate``, go to ``dst``: a cache of ``layout`` TND, BBND
    or BNBD, or with "ROWS" [T, H, ...] (the queries).  ``dst``'s type says how
    they are stored; int8 and uint8 (MXFP4) take ``scale``."""
    src: torch.Tensor
    dst: torch.Tensor
    layout: object
    scale: Optional[torch.Tensor] = None
    rotate: bool = False


# msa_tensor_t packed by hand (data, dtype, ndim, shape[4], stride[4]): a step
# of small calls is bound by the host, and filling a ctypes structure field by
# field costs several times as much as packing its bytes
_FIELDS = {n: "Qii%dq%dx%dq%dx" % (n, 32 - 8 * n, n, 32 - 8 * n) for n in range(1, 5)}
_PACK = {n: struct.Struct("<" + f).pack for n, f in _FIELDS.items()}
# msa_append_item_t: src, dst, scale, layout, rotate
_PACK_ITEM = {(i, j): struct.Struct("<" + f + g + "Qii").pack
              for i, f in _FIELDS.items() for j, g in _FIELDS.items()}


def _packed(t: torch.Tensor) -> bytes:
    stride = t.stride()
    n = len(stride)
    if not 1 <= n <= 4:
        raise ValueError(f"a tensor of {n} axes: 1 to 4 are taken")
    return _PACK[n](t.data_ptr(), DTYPE_CODE.get(t.dtype, -1), n, *t.shape, *stride)


def _address(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _check_lengths(cu_seqlens_q, kv_len, block_table, max_blocks, paged) -> int:
    """The request count B, from tensors whose extents the C ABI takes on trust."""
    i32 = torch.int32
    if cu_seqlens_q.dtype != i32 or not cu_seqlens_q.is_contiguous():
        raise ValueError("cu_seqlens_q must be a contiguous int32 tensor")
    if kv_len.dtype != i32 or not kv_len.is_contiguous():
        raise ValueError("kv_len must be a contiguous int32 tensor")
    if kv_len.dim() != 1:
        raise ValueError("kv_len must be 1-D [B] (per-request lengths)")
    B = kv_len.numel()
    if cu_seqlens_q.dim() != 1 or cu_seqlens_q.numel() != B + 1:
        raise ValueError(f"cu_seqlens_q must be [B+1] = [{B + 1}], got "
                         f"{tuple(cu_seqlens_q.shape)}")
    if block_table is None:
        if paged:
            raise ValueError("paged layouts need a block_table")
        return B
    if block_table.dtype != i32 or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous int32 tensor")
    shape = block_table.shape
    if paged and (len(shape) != 2 or shape[0] < B or shape[1] != max_blocks):
        raise ValueError(f"block_table must be [>= {B}, max_blocks = {max_blocks}], got "
                         f"{tuple(shape)}")
    return B


def _stream_of(handle, dev):
    """The torch stream of a raw handle (0: the device's default stream)."""
    if not handle:
        return torch.cuda.default_stream(dev)
    return torch.cuda.ExternalStream(handle, device=dev)


# torch's getter of the current stream's handle, where this build of torch has it
_current_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream, index: int):
    """``_stream_handle`` without a stream object for the current stream, which
    costs a small call a microsecond (torch's own compiled code takes the handle
    the same way; a torch without that getter costs the stream object)."""
    if stream is None and index >= 0 and _current_raw is not None:
        return _current_raw(index)
    return _stream_handle(stream, index)


def _guard(index: int):
    """Makes the tensors' device current for a launch, where it is not."""
    if index < 0 or torch.cuda.current_device() == index:
        return _NO_GUARD
    return torch.cuda.device(index)


_NO_GUARD = contextlib.nullcontext()


_ITEM_LAYOUT = {**LAYOUT_CODE, "ROWS": ROWS}


def _item_layout(layout) -> int:
    if isinstance(layout, str):
        return _ITEM_LAYOUT.get(layout.upper(), -1)
    return int(layout)


def _check_axes(axis_positions, pair_axes, lead, index, rotary) -> bytes:
    """The axis of each pair as bytes, of tensors that fit the items."""
    if (axis_positions.dtype != torch.int32 or not axis_positions.is_contiguous() or
            axis_positions.dim() != 2 or axis_positions.shape[1] != lead.shape[0]):
        raise ValueError(f"axis_positions must be a contiguous int32 [axes, {lead.shape[0]}] "
                         f"tensor, got {axis_positions.dtype} {tuple(axis_positions.shape)}")
    if axis_positions.get_device() != index:
        raise ValueError(f"tensors are on {axis_positions.device} and {lead.device}")
    if pair_axes is None or len(pair_axes) != rotary // 2:
        raise ValueError(f"pair_axes must hold the axis of each of the {rotary // 2} pairs")
    try:
        # (an array's own bytes would be those of its wider integers)
        return bytes(pair_axes if isinstance(pair_axes, (bytes, list, tuple)) else
                     [operator.index(x) for x in pair_axes])
    except (TypeError, ValueError) as e:
        raise ValueError("pair_axes must hold integers from 0 on") from e


def msa_cache_append(items: Sequence[CacheItem], cos: Optional[torch.Tensor],
                     sin: Optional[torch.Tensor], block_table: Optional[torch.Tensor],
                     cu_seqlens_q: torch.Tensor, kv_len: torch.Tensor,
                     interleaved: bool = False, stream=None, block_size: int = BLOCK_SIZE,
                     axis_positions: Optional[torch.Tensor] = None,
                     pair_axes: Optional[Sequence[int]] = None) -> None:
    """Append the new tokens' rows to their caches, rotated by their positions
    and encoded as the caches hold them, and rotate or encode the queries, in
    one launch (see ``CacheItem``; the C ABI's header defines the encodings).

    ``cos`` and ``sin`` [positions, rotary_dim / 2] float32 may be None if no
    item is rotated, ``block_table`` [>= B, MB] int32 if no item is paged;
    ``kv_len`` counts the new tokens.

    With ``axis_positions`` ([axes, T] int32, 1 to 4 axes) pair r of a token is
    rotated by the position of axis ``pair_axes[r]`` (rotary_dim / 2 integers, or
    the same as bytes) instead of the token's position in its sequence; if no item
    is rotated, neither is looked at."""
    lib = _lib or load_library()
    if not 1 <= len(items) <= APPEND_MAX_ITEMS:
        raise ValueError(f"1 to {APPEND_MAX_ITEMS} items, got {len(items)}")
    lead = items[0][0]
    index = lead.get_device()
    for t in (cos, sin, block_table, cu_seqlens_q, kv_len):
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors are on {t.device} and {lead.device}")
    paged = block_table is not None
    max_blocks = block_table.shape[-1] if paged else 0
    B = _check_lengths(cu_seqlens_q, kv_len, block_table, max_blocks, paged)
    positions = rotary = 0
    rotated = any(it[4] for it in items)
    if cos is not None and sin is not None:
        if cos.shape != sin.shape or cos.dim() != 2:
            raise ValueError("cos and sin must both be [positions, rotary_dim / 2]")
        for name, t in (("cos", cos), ("sin", sin)):
            if t.dtype != torch.float32 or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous float32 tensor")
        positions, rotary = cos.shape[0], 2 * cos.shape[1]
    elif cos is not None or sin is not None or rotated:
        raise ValueError("rotated items need both cos and sin")
    axes = None
    if axis_positions is not None and rotated:
        axes = _check_axes(axis_positions, pair_axes, lead, index, rotary)
    elif pair_axes is not None and rotated:
        raise ValueError("pair_axes needs axis_positions")
    packed, code = [], DTYPE_CODE.get
    for i, (src, dst, layout, scale, rotate) in enumerate(items):
        lay = _ITEM_LAYOUT.get(layout)
        if lay is None:
            lay = _item_layout(layout)
        if src.get_device() != index or dst.get_device() != index:
            raise ValueError(f"item {i}: src is on {src.device}, dst on {dst.device}")
        if lay in (1, 2) and not paged:
            raise ValueError(f"item {i}: paged layouts need a block_table")
        at = 0
        if scale is not None:
            i8 = dst.dtype == torch.int8
            want = torch.float32 if i8 else torch.uint8
            n = dst.numel() // (128 if i8 else 16)
            if (scale.dtype != want or not scale.is_contiguous() or scale.numel() != n or
                    scale.get_device() != index):
                raise ValueError(f"item {i}: scale must be a contiguous {want} tensor of {n} "
                                 f"elements beside dst, got {scale.dtype} "
                                 f"{tuple(scale.shape)} on {scale.device}")
            at = scale.data_ptr()
        m, n = len(src.shape), len(dst.shape)
        if not (1 <= m <= 4 and 1 <= n <= 4):
            raise ValueError(f"item {i}: src has {m} axes, dst {n}: 1 to 4 are taken")
        packed.append(_PACK_ITEM[m, n](
            src.data_ptr(), code(src.dtype, -1), m, *src.shape, *src.stride(),
            dst.data_ptr(), code(dst.dtype, -1), n, *dst.shape, *dst.stride(),
            at, lay, 1 if rotate else 0))
    if index < 0 and lead.numel():
        raise ValueError(f"the tensors must be on a GPU, src is on {lead.device}")
    handle = _raw_stream(stream, index)
    head = (b"".join(packed), len(items), _address(cos), _address(sin), positions, rotary,
            1 if interleaved else 0)
    tail = (_address(block_table), max_blocks, cu_seqlens_q.data_ptr(), kv_len.data_ptr(), B,
            int(block_size), handle)
    with _guard(index):
        if axes is None:
            st = lib.msa_cache_append(*head, *tail)
        else:
            st = lib.msa_cache_append_axes(*head, axis_positions.data_ptr(),
                                           axis_positions.shape[0], axes, *tail)
    if st:
        _raise_status(st)


def msa_attention_workspace(T: int, batch: int, Hq: int, Hkv: int, max_blocks: int,
                            num_blocks: int = 0) -> int:
    """Bytes of workspace that an attention call of these sizes needs
    (``num_blocks`` 0: dense)."""
    return int(load_library().msa_attention_workspace(int(T), int(batch), int(Hq), int(Hkv),
                                                      int(max_blocks), int(num_blocks)))


def msa_attention_tile_rows(T: int, batch: int, Hq: int, Hkv: int, max_blocks: int,
                            num_blocks: int = 0) -> int:
    """Rows of the tiles (16, 128 or 256) that an attention call of these sizes
    uses (``num_blocks`` 0: dense)."""
    return int(load_library().msa_attention_tile_rows(int(T), int(batch), int(Hq), int(Hkv),
                                                      int(max_blocks), int(num_blocks)))


def msa_attention_ex_workspace(T: int, batch: int, Hq: int, Hkv: int, max_blocks: int) -> int:
    """Bytes of workspace with which an attention call of these sizes with
    ``softcap``, ``slopes`` or ``visible`` is split as it would choose to
    (``msa_attention_workspace``, or more)."""
    return int(load_library().msa_attention_ex_workspace(int(T), int(batch), int(Hq), int(Hkv),
                                                         int(max_blocks)))


_workspace_bytes = functools.lru_cache(maxsize=1024)(msa_attention_workspace)
_form_workspace_bytes = functools.lru_cache(maxsize=1024)(msa_attention_ex_workspace)


def _attention(query, key, value, blocks, block_table, cu_seqlens_q, kv_len, layout, sparse_mode,
               softmax_scale, out, lse, max_blocks, workspace, stream, block_size, softcap=0.0,
               slopes=None, visible=None):
    lib = _lib or load_library()
    index = query.get_device()
    if (key.get_device() != index or value.get_device() != index or
            cu_seqlens_q.get_device() != index or kv_len.get_device() != index or
            out.get_device() != index or
            (block_table is not None and block_table.get_device() != index) or
            (lse is not None and lse.get_device() != index) or
            (blocks is not None and blocks.get_device() != index) or
            (workspace is not None and workspace.get_device() != index)):
        raise ValueError(f"every tensor must be on the query's device, {query.device}")
    lay = _layout_code(layout)
    max_blocks = int(max_blocks)
    B = _check_lengths(cu_seqlens_q, kv_len, block_table, max_blocks, lay in (1, 2))
    shape = query.shape
    if len(shape) != 3:
        raise ValueError(f"query must be [T, Hq, 128], got {tuple(shape)}")
    T, Hq, D = shape
    if out.dtype != query.dtype or out.shape != shape or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {query.dtype} {tuple(shape)} tensor")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != shape[:2] or
                            not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous float32 [{T}, {Hq}] tensor")
    if key.dim() == 4:
        Hkv = key.shape[1 if lay == 2 else 2]
    else:                                # packed, or one head with no axis of its own
        kr = _key_rows(key, lay)
        Hkv = kr[1] if kr is not None else 0
    k = 0
    if blocks is not None:
        if (blocks.dtype != torch.int32 or not blocks.is_contiguous() or blocks.dim() != 3 or
                tuple(blocks.shape[:2]) != (T, Hkv)):
            raise ValueError(f"blocks must be a contiguous int32 [{T}, {Hkv}, k] tensor, got "
                             f"{blocks.dtype} {tuple(blocks.shape)}")
        k = blocks.shape[2]
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if slopes is not None and (slopes.dtype != torch.float32 or slopes.shape != (Hq,) or
                               not slopes.is_contiguous() or slopes.get_device() != index):
        raise ValueError(f"slopes must be a contiguous float32 [{Hq}] tensor on {query.device}, "
                         f"got {slopes.dtype} {tuple(slopes.shape)} on {slopes.device}")
    if visible is not None and (visible.dtype != torch.int32 or visible.shape != (T, 2) or
                                not visible.is_contiguous() or visible.get_device() != index):
        raise ValueError(f"visible must be a contiguous int32 [{T}, 2] tensor on {query.device}, "
                         f"got {visible.dtype} {tuple(visible.shape)} on {visible.device}")
    if index < 0 and query.numel():
        raise ValueError(f"the tensors must be on a GPU, query is on {query.device}")
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    handle = _raw_stream(stream, index)
    with _guard(index):
        form = softcap or slopes is not None or visible is not None
        need = (0 if workspace is not None else
                _form_workspace_bytes(T, B, Hq, Hkv, max_blocks) if form else
                _workspace_bytes(T, B, Hq, Hkv, max_blocks, k))
        if need:
            # memory of the stream that the kernels run on, so that it is
            # handed on only behind them
            if stream is None:
                workspace = query.new_empty(need, dtype=torch.uint8)
            else:
                with torch.cuda.stream(_stream_of(handle, query.device)):
                    workspace = query.new_empty(need, dtype=torch.uint8)
        wb = 0 if workspace is None else workspace.numel() * workspace.element_size()
        lens = (_address(block_table), max_blocks, cu_seqlens_q.data_ptr(), kv_len.data_ptr(), B,
                int(block_size), lay, int(sparse_mode), scale)
        rest = (out.data_ptr(), _address(lse), _address(workspace), wb, handle)
        if blocks is not None:
            st = lib.msa_block_attention(_packed(query), _packed(key), _packed(value),
                                         blocks.data_ptr(), k, *lens, *rest)
        elif form:
            st = lib.msa_attention_ex(_packed(query), _packed(key), _packed(value), *lens,
                                      float(softcap or 0.0), _address(slopes), _address(visible),
                                      *rest)
        else:
            st = lib.msa_attention(_packed(query), _packed(key), _packed(value), *lens, *rest)
    if st:
        _raise_status(st)
    return out


def msa_attention(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                  block_table: Optional[torch.Tensor], cu_seqlens_q: torch.Tensor,
                  kv_len: torch.Tensor, layout, sparse_mode: int, softmax_scale: Optional[float],
                  out: torch.Tensor, max_blocks: int, lse: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None,
                  block_size: int = BLOCK_SIZE, softcap: Optional[float] = None,
                  slopes: Optional[torch.Tensor] = None,
                  visible: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Call the C ABI: ``out`` ([T, Hq, 128], the query's type) receives the
    attention of every new token over its request's visible keys, ``lse``
    ([T, Hq] float32, if given) the log of its softmax's sum; asynchronous on
    ``stream`` (default: torch's current stream).  ``softmax_scale`` None is
    1 / sqrt(128).  Without ``workspace`` the memory that a split over the keys
    needs (``msa_attention_workspace``; with one of the following
    ``msa_attention_ex_workspace``) is allocated here.

    ``softcap`` (None or 0: none) caps the scores by softcap * tanh(S / softcap);
    ``slopes`` ([Hq] float32) takes slopes[h] * |position - key| off them;
    ``visible`` ([T, 2] int32: first key and end of keys) narrows what each token
    sees beyond ``sparse_mode`` (documents with mode 3, images and prefixes with
    mode 0)."""
    return _attention(query, key, value, None, block_table, cu_seqlens_q, kv_len, layout,
                      sparse_mode, softmax_scale, out, lse, max_blocks, workspace, stream,
                      block_size, softcap, slopes, visible)


def msa_block_attention(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                        blocks: torch.Tensor, block_table: Optional[torch.Tensor],
                        cu_seqlens_q: torch.Tensor, kv_len: torch.Tensor, layout,
                        sparse_mode: int, softmax_scale: Optional[float], out: torch.Tensor,
                        max_blocks: int, lse: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None,
                        block_size: int = BLOCK_SIZE) -> torch.Tensor:
    """``msa_attention`` over the blocks that ``blocks`` ([T, Hkv, k] int32, as
    ``msa_block_topk`` writes them) names for each token and KV head."""
    if blocks is None:
        raise ValueError("blocks is required")
    return _attention(query, key, value, blocks, block_table, cu_seqlens_q, kv_len, layout,
                      sparse_mode, softmax_scale, out, lse, max_blocks, workspace, stream,
                      block_size)


def _outputs(query, return_lse, stream):
    """out and lse of a call that leaves them to the binding; those of a call on
    a given stream belong to that stream, as its workspace does."""
    if stream is not None and query.is_cuda:
        with torch.cuda.stream(_stream_of(_stream_handle(stream, query.device), query.device)):
            return _outputs(query, return_lse, None)
    shape = query.shape
    if len(shape) != 3:
        raise ValueError(f"query must be [T, Hq, 128], got {tuple(shape)}")
    out = torch.empty_like(query, memory_format=torch.contiguous_format)
    if not return_lse:
        return out, None
    return out, query.new_empty((shape[0], shape[1]), dtype=torch.float32)


def _default_blocks(key, block_table) -> int:
    """max_blocks where the caller leaves it out: the table's width, or as many
    as all packed keys would fill."""
    return block_table.shape[-1] if block_table is not None else (key.shape[0] + 127) // 128


def attention(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
              block_table: Optional[torch.Tensor], cu_seqlens_q: torch.Tensor,
              kv_len: torch.Tensor, layout, sparse_mode: int = 3,
              softmax_scale: Optional[float] = None, max_blocks: Optional[int] = None,
              return_lse: bool = False, stream=None, softcap: Optional[float] = None,
              slopes: Optional[torch.Tensor] = None, visible: Optional[torch.Tensor] = None):
    """Allocate ``out`` (and ``lse``) and fill them with ``msa_attention`` (which
    says what ``softcap``, ``slopes`` and ``visible`` do);
    returns ``out`` or ``(out, lse)``.  Rows that no request holds (a padded
    batch) are not written.  On a ``stream`` that is given, they are that
    stream's memory: use on another stream needs an ordering, and ``record_stream``
    before they are freed."""
    out, lse = _outputs(query, return_lse, stream)
    if max_blocks is None:
        max_blocks = _default_blocks(key, block_table)
    _attention(query, key, value, None, block_table, cu_seqlens_q, kv_len, layout, sparse_mode,
               softmax_scale, out, lse, max_blocks, None, stream, BLOCK_SIZE, softcap, slopes,
               visible)
    return (out, lse) if return_lse else out


def block_attention(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                    blocks: torch.Tensor, block_table: Optional[torch.Tensor],
                    cu_seqlens_q: torch.Tensor, kv_len: torch.Tensor, layout,
                    sparse_mode: int = 3, softmax_scale: Optional[float] = None,
                    max_blocks: Optional[int] = None, return_lse: bool = False, stream=None):
    """Allocate ``out`` (and ``lse``) and fill them with
    ``msa_block_attention``, as ``attention`` does; returns ``out`` or
    ``(out, lse)``."""
    if blocks is None:
        raise ValueError("blocks is required")
    out, lse = _outputs(query, return_lse, stream)
    if max_blocks is None:
        max_blocks = _default_blocks(key, block_table)
    _attention(query, key, value, blocks, block_table, cu_seqlens_q, kv_len, layout, sparse_mode,
               softmax_scale, out, lse, max_blocks, None, stream, BLOCK_SIZE)
    return (out, lse) if return_lse else out


# ---------------------------------------------------------------------------
# the step's tables
# ---------------------------------------------------------------------------


class StepTables(NamedTuple):
    """What ``msa_step_tables`` writes: int32 tensors, but int64 slots."""
    cu_seqlens_q: torch.Tensor   # [B + 1]
    kv_len: torch.Tensor         # [B], new tokens included
    start_loc: torch.Tensor      # [B], block of the first new token
    block_table: torch.Tensor    # [B, max_blocks]
    positions: torch.Tensor      # [T]
    slots: torch.Tensor          # [T], page * 128 + position % 128, -1: none
    cu_pages: torch.Tensor       # [B + 1], pages taken from the free list


def new_step_tables(batch: int, T: int, max_blocks: int, device=None) -> StepTables:
    """Tensors for ``msa_step_tables`` to write, which a server keeps from step
    to step."""
    def ints(*shape):
        return torch.empty(shape, dtype=torch.int32, device=device)

    return StepTables(ints(batch + 1), ints(batch), ints(batch), ints(batch, max_blocks), ints(T),
                      torch.empty(T, dtype=torch.int64, device=device), ints(batch + 1))


_TABLE_ARGS = ("new_tokens", "ctx_len", "rows", "pool", "free_pages", "free_count", "free_out",
               "cu_seqlens_q", "kv_len", "start_loc", "block_table", "positions", "cu_pages")


def msa_step_tables(new_tokens: torch.Tensor, ctx_len: torch.Tensor, pool: torch.Tensor,
                    free_pages: torch.Tensor, free_count: torch.Tensor, out: StepTables,
                    rows: Optional[torch.Tensor] = None, free_out: Optional[torch.Tensor] = None,
                    stream=None, block_size: int = BLOCK_SIZE) -> StepTables:
    """Call the C ABI: from ``new_tokens`` and ``ctx_len`` ([B] int32) the tables
    of one step, into ``out``; blocks that the new tokens begin take pages from
    the end of ``free_pages``' first ``free_count[0]``, and are entered in
    ``pool`` ([rows, blocks] int32), whose row ``rows[b]`` (None: b) is request
    b's.  ``free_out`` ([2] int32: pages left, pages missing) is ``free_count``
    itself if it is None.  T and max_blocks are ``out``'s; asynchronous on
    ``stream`` (default: torch's current stream)."""
    lib = _lib or load_library()
    index = new_tokens.get_device()
    if free_out is None:
        free_out = free_count
    cu, kv, start, table, positions, slots, pages = out
    B, T = new_tokens.numel(), positions.numel()
    if pool.dim() != 2 or table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError(f"pool must be [rows, blocks], block_table [{B}, max_blocks] and "
                         f"free_pages 1-D, got {tuple(pool.shape)}, {tuple(table.shape)} and "
                         f"{tuple(free_pages.shape)}")
    max_blocks = table.shape[1]
    # (a step of few requests is bound by the host: elements are counted, which a
    # compact tensor's shape adds nothing to)
    i32, n, free = torch.int32, B + 1, free_pages.numel()
    pool_rows, pool_blocks = pool.shape
    for i, (t, size) in enumerate(((new_tokens, B), (ctx_len, B), (rows, B),
                                   (pool, pool_rows * pool_blocks), (free_pages, free),
                                   (free_count, 2), (free_out, 2), (cu, n), (kv, B), (start, B),
                                   (table, B * max_blocks), (positions, T), (pages, n))):
        if t is not None and (t.dtype is not i32 or t.numel() != size or
                              not t.is_contiguous() or t.get_device() != index):
            raise ValueError(f"{_TABLE_ARGS[i]} must be a contiguous int32 tensor of {size} "
                             f"elements on {new_tokens.device}, got {t.dtype} {tuple(t.shape)} "
                             f"on {t.device}")
    if (slots.dtype is not torch.int64 or slots.numel() != T or not slots.is_contiguous() or
            slots.get_device() != index):
        raise ValueError(f"slots must be a contiguous int64 tensor of {T} elements on "
                         f"{new_tokens.device}, got {slots.dtype} {tuple(slots.shape)} on "
                         f"{slots.device}")
    if index < 0:
        raise ValueError(f"the tensors must be on a GPU, new_tokens is on {new_tokens.device}")
    handle = _raw_stream(stream, index)
    with _guard(index):
        st = lib.msa_step_tables(
            new_tokens.data_ptr(), ctx_len.data_ptr(), _address(rows), B, pool.data_ptr(),
            pool_rows, pool_blocks, free_pages.data_ptr(), free, free_count.data_ptr(),
            free_out.data_ptr(), max_blocks, T, int(block_size), cu.data_ptr(), kv.data_ptr(),
            start.data_ptr(), table.data_ptr(), positions.data_ptr(), slots.data_ptr(),
            pages.data_ptr(), handle)
    if st:
        _raise_status(st)
    return out


def step_tables(new_tokens: torch.Tensor, ctx_len: torch.Tensor, pool: torch.Tensor,
                free_pages: torch.Tensor, free_count: torch.Tensor, T: int,
                rows: Optional[torch.Tensor] = None, max_blocks: Optional[int] = None,
                free_out: Optional[torch.Tensor] = None, stream=None) -> StepTables:
    """Allocate the tables of a step of up to ``T`` new tokens and fill them with
    ``msa_step_tables`` (``max_blocks`` defaults to the pool's width).  On a
    ``stream`` that is given, they are that stream's memory, as ``attention``'s
    outputs are."""
    width = pool.shape[-1] if max_blocks is None else max_blocks
    if stream is not None and new_tokens.is_cuda:
        with torch.cuda.stream(_stream_of(_stream_handle(stream, new_tokens.device),
                                          new_tokens.device)):
            out = new_step_tables(new_tokens.numel(), T, width, new_tokens.device)
    else:
        out = new_step_tables(new_tokens.numel(), T, width, new_tokens.device)
    return msa_step_tables(new_tokens, ctx_len, pool, free_pages, free_count, out, rows=rows,
                           free_out=free_out, stream=stream)
