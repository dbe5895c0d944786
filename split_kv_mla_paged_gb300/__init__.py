"""Paged FP8 MLA split-KV decode for GB300 (sm_103a).

A thin ctypes binding over libmla_decode.so (declared in include/mla_decode.h).
The functions keep the C names and only marshal arguments: every step of the
decode runs in the library's CUDA kernels.  PyTorch supplies device memory and
streams.  There is no fallback: if the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import dataclasses
import operator
import os
import threading
from typing import Optional, Sequence

import numpy as np

from . import build as _build

__all__ = [
    "MLA_OK", "MLA_ERR_INVALID_ARG", "MLA_ERR_UNSUPPORTED", "MLA_ERR_WORKSPACE_TOO_SMALL",
    "MLA_ERR_CUDA", "MLA_ERR_TIMEOUT", "MlaError", "Plan", "load_library", "library_path",
    "mla_decode_plan", "mla_decode_workspace_size", "mla_decode_workspace_init", "mla_decode",
    "mla_decode_splitkv", "mla_decode_merge", "mla_merge", "mla_decode_status", "mla_last_error",
    "mla_decode_static_ws", "mla_decode_static_ws_status", "mla_kv_append", "mla_decode_ex",
    "mla_decode_bf16", "mla_decode_sparse", "mla_decode_plan_items", "mla_decode_bf16_ex",
    "mla_decode_bf16_sparse", "mla_decode_plan_items_bf16", "DecodeOptions",
    "decode", "merge", "MLA_ERR_NO_PAGES", "CACHE_FP8", "CACHE_BF16", "CACHE_FP4",
    "FP4_PAGE_BYTES", "mla_decode_fp4", "mla_decode_fp4_sparse", "PrologueArgs", "mla_prologue", "mla_pages_copy", "mla_pages_remap",
    "PagePool", "copy_pages", "fp4_pool",
    "EXPORTED_SYMBOLS",
]

MLA_OK = 0
MLA_ERR_INVALID_ARG = 1
MLA_ERR_UNSUPPORTED = 2
MLA_ERR_WORKSPACE_TOO_SMALL = 3
MLA_ERR_CUDA = 4
MLA_ERR_TIMEOUT = 5
MLA_ERR_NO_PAGES = 6
_STATUS_NAMES = {
    0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED",
    3: "MLA_ERR_WORKSPACE_TOO_SMALL", 4: "MLA_ERR_CUDA", 5: "MLA_ERR_TIMEOUT",
    6: "MLA_ERR_NO_PAGES",
}
EXPORTED_SYMBOLS = ("mla_decode_plan", "mla_decode_workspace_size", "mla_decode_workspace_init",
                    "mla_decode", "mla_decode_splitkv", "mla_decode_merge", "mla_merge",
                    "mla_decode_status", "mla_last_error", "mla_debug_set_wait_limit",
                    "mla_decode_static_ws", "mla_decode_static_ws_status", "mla_kv_append",
                    "mla_decode_ex", "mla_decode_bf16", "mla_decode_sparse",
                    "mla_decode_plan_items", "mla_decode_bf16_ex", "mla_decode_bf16_sparse",
                    "mla_decode_plan_items_bf16", "mla_debug_set_expire", "mla_prologue",
                    "mla_decode_fp4", "mla_decode_fp4_sparse",
                    "mla_pages_copy", "mla_pages_remap", "mla_pool_create", "mla_pool_destroy",
                    "mla_pool_free_pages", "mla_pool_references", "mla_pool_alloc",
                    "mla_pool_release", "mla_pool_fork", "mla_pool_compact")

HEAD_DIM = 576
LATENT_DIM = 512
ROPE_DIM = 64
PAGE_SIZE = 32
TILE_TOKENS = 128
MAX_SPLITS = 256
PAGES_SPLIT_CAP = 128
# Kinds of paged cache (mla_decode.h: MLA_CACHE_*) and the bytes of a 4-bit page.
CACHE_FP8, CACHE_BF16, CACHE_FP4 = 0, 1, 2
FP4_BLOCK = 32
FP4_PAGE_BYTES = 10752


class DecodeOptions(ctypes.Structure):
    """mla_decode_options_t (include/mla_decode.h)."""
    _fields_ = [("q_scale_dev", ctypes.c_void_p), ("kv_scale_dev", ctypes.c_void_p),
                ("softmax_scale_dev", ctypes.c_void_p), ("output_scale", ctypes.c_float),
                ("sinks", ctypes.c_void_p), ("query_lens", ctypes.c_void_p),
                ("kv_bounds", ctypes.c_void_p), ("cta_items", ctypes.c_void_p),
                ("num_ctas", ctypes.c_int32), ("persistent_ctas", ctypes.c_int32),
                ("phases", ctypes.c_int32)]


class PrologueArgs(ctypes.Structure):
    """mla_prologue_args_t (include/mla_decode.h)."""
    _fields_ = [("n_tokens", ctypes.c_int64), ("positions", ctypes.c_void_p),
                ("cos_sin", ctypes.c_void_p), ("rope_positions", ctypes.c_void_p),
                ("rope_rows", ctypes.c_int32), ("rope_halves", ctypes.c_int32),
                ("kv_rows", ctypes.c_void_p), ("kv_row_stride", ctypes.c_int64),
                ("norm_weight", ctypes.c_void_p), ("norm_eps", ctypes.c_float),
                ("max_pages_per_req", ctypes.c_int32), ("req_idx", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("kv_pages", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("batch", ctypes.c_int32),
                ("cache_kind", ctypes.c_int32), ("kv_scale", ctypes.c_float),
                ("q_scale", ctypes.c_float), ("q_rows", ctypes.c_void_p),
                ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("q_out", ctypes.c_void_p), ("num_heads", ctypes.c_int32),
                ("q_kind", ctypes.c_int32), ("status", ctypes.c_void_p)]


# mla_decode_options_t.phases: both phases, the split-KV kernel only, the merge only.
PHASE_ALL, PHASE_SPLIT, PHASE_MERGE = 0, 1, 2


class MlaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


_lock = threading.Lock()
_lib: Optional[ctypes.CDLL] = None


def library_path() -> str:
    return _build.LIB_PATH


def load_library() -> ctypes.CDLL:
    """Load libmla_decode.so (built by `build.build()`); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with split_kv_mla_paged_gb300.build.build() "
                "(there is no fallback implementation)")
        lib = ctypes.CDLL(path)
        vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                                 ctypes.c_size_t)
        lib.mla_decode_plan.restype = ctypes.c_int
        lib.mla_decode_plan.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, vp, vp]
        for name in ("mla_decode_plan_items", "mla_decode_plan_items_bf16"):
            getattr(lib, name).restype = ctypes.c_int
            getattr(lib, name).argtypes = [vp, i32, i32, i32, vp, i32, vp]
        lib.mla_decode_workspace_size.restype = sz
        lib.mla_decode_workspace_size.argtypes = [i32, i32, i32, i32]
        dec_args = [vp, vp, i64, vp, i32, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, f32, f32,
                    vp, sz, vp, vp, vp, vp]
        for name in ("mla_decode", "mla_decode_splitkv", "mla_decode_merge"):
            getattr(lib, name).restype = ctypes.c_int
            getattr(lib, name).argtypes = dec_args
        lib.mla_decode_ex.restype = ctypes.c_int
        lib.mla_decode_ex.argtypes = dec_args[:-1] + [ctypes.POINTER(DecodeOptions), vp]
        lib.mla_decode_sparse.restype = ctypes.c_int
        lib.mla_decode_sparse.argtypes = (dec_args[:6] + [vp, i32] + dec_args[6:-1]
                                          + [ctypes.POINTER(DecodeOptions), vp])
        lib.mla_decode_fp4.restype = ctypes.c_int
        lib.mla_decode_fp4.argtypes = lib.mla_decode_ex.argtypes
        lib.mla_decode_fp4_sparse.restype = ctypes.c_int
        lib.mla_decode_fp4_sparse.argtypes = lib.mla_decode_sparse.argtypes
        lib.mla_decode_bf16.restype = ctypes.c_int
        lib.mla_decode_bf16.argtypes = dec_args[:14] + [f32] + dec_args[17:]
        lib.mla_decode_bf16_ex.restype = ctypes.c_int
        lib.mla_decode_bf16_ex.argtypes = (dec_args[:14] + [f32] + dec_args[17:-1]
                                           + [ctypes.POINTER(DecodeOptions), vp])
        lib.mla_decode_bf16_sparse.restype = ctypes.c_int
        lib.mla_decode_bf16_sparse.argtypes = (dec_args[:6] + [vp, i32] + dec_args[6:14] + [f32]
                                               + dec_args[17:-1]
                                               + [ctypes.POINTER(DecodeOptions), vp])
        lib.mla_decode_workspace_init.restype = ctypes.c_int
        lib.mla_decode_workspace_init.argtypes = [vp, sz, vp]
        lib.mla_merge.restype = ctypes.c_int
        lib.mla_merge.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp, vp]
        lib.mla_decode_status.restype = ctypes.c_int
        lib.mla_decode_status.argtypes = [vp, vp]
        lib.mla_decode_static_ws.restype = ctypes.c_int
        lib.mla_decode_static_ws.argtypes = [vp, vp, i64, vp, i32, vp, vp, vp, i32, i32, i32, i32,
                                             i32, i32, f32, f32, f32, vp, vp, vp, vp]
        lib.mla_decode_static_ws_status.restype = ctypes.c_int
        lib.mla_decode_static_ws_status.argtypes = [vp]
        lib.mla_kv_append.restype = ctypes.c_int
        lib.mla_kv_append.argtypes = [vp, i64, vp, vp, vp, i32, i32, vp, i64, f32, vp, vp]
        lib.mla_prologue.restype = ctypes.c_int
        lib.mla_prologue.argtypes = [ctypes.POINTER(PrologueArgs), vp]
        lib.mla_pages_copy.restype = ctypes.c_int
        lib.mla_pages_copy.argtypes = [vp, i64, i32, vp, i64, i32, vp, vp, vp, i64, vp, vp]
        lib.mla_pages_remap.restype = ctypes.c_int
        lib.mla_pages_remap.argtypes = [vp, i64, vp, i64, vp, vp]
        lib.mla_pool_create.restype = ctypes.c_int
        lib.mla_pool_create.argtypes = [i64, ctypes.POINTER(vp)]
        lib.mla_pool_destroy.restype = None
        lib.mla_pool_destroy.argtypes = [vp]
        lib.mla_pool_free_pages.restype = i64
        lib.mla_pool_free_pages.argtypes = [vp]
        lib.mla_pool_references.restype = i64
        lib.mla_pool_references.argtypes = [vp, i32]
        lib.mla_pool_alloc.restype = ctypes.c_int
        lib.mla_pool_alloc.argtypes = [vp, i64, vp]
        lib.mla_pool_release.restype = ctypes.c_int
        lib.mla_pool_release.argtypes = [vp, vp, i64]
        lib.mla_pool_fork.restype = ctypes.c_int
        lib.mla_pool_fork.argtypes = [vp, vp, i64, i64, vp, vp, vp, vp, vp]
        lib.mla_pool_compact.restype = ctypes.c_int
        lib.mla_pool_compact.argtypes = [vp, i64, vp, vp, vp, vp]
        lib.mla_debug_set_wait_limit.restype = None
        lib.mla_debug_set_wait_limit.argtypes = [ctypes.c_longlong]
        lib.mla_debug_set_expire.restype = None
        lib.mla_debug_set_expire.argtypes = [i32, i32]
        lib.mla_last_error.restype = ctypes.c_char_p
        lib.mla_last_error.argtypes = []
        _lib = lib
        return lib


def mla_last_error() -> str:
    return load_library().mla_last_error().decode("utf-8", "replace")


def _check(status: int) -> None:
    if status != MLA_OK:
        raise MlaError(status, mla_last_error())


def _ptr(t) -> Optional[int]:
    """Address of a torch tensor / numpy array, or None."""
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


@dataclasses.dataclass
class Plan:
    splits: np.ndarray   # int32 [B]
    chunks: np.ndarray   # int32 [B]
    kv_split: int
    workspace_bytes: int

    @property
    def max_splits(self) -> int:
        return int(self.splits.max())


def mla_decode_plan(kv_lens: Sequence[int], num_heads: int, q_len: int, sm_count: int = 0,
                    target_ctas: int = 0) -> Plan:
    lib = load_library()
    lens = np.ascontiguousarray(np.asarray(kv_lens, dtype=np.int32))
    b = int(lens.shape[0])
    splits = np.zeros(b, dtype=np.int32)
    chunks = np.zeros(b, dtype=np.int32)
    kvs = ctypes.c_int32(0)
    ws = ctypes.c_size_t(0)
    _check(lib.mla_decode_plan(lens.ctypes.data, b, int(num_heads), int(q_len), int(sm_count),
                               int(target_ctas), splits.ctypes.data, chunks.ctypes.data,
                               ctypes.addressof(kvs), ctypes.addressof(ws)))
    return Plan(splits=splits, chunks=chunks, kv_split=int(kvs.value), workspace_bytes=int(ws.value))


def mla_decode_plan_items(splits, num_heads: int, q_len: int, bf16: bool = False) -> np.ndarray:
    """CTA item list of a plan (one int32 per CTA that has work, split-major);
    bf16=True builds it with the BF16 kernels' row groups."""
    lib = load_library()
    fn = lib.mla_decode_plan_items_bf16 if bf16 else lib.mla_decode_plan_items
    sp = np.ascontiguousarray(np.asarray(splits, dtype=np.int32))
    n = ctypes.c_int32(0)
    _check(fn(sp.ctypes.data, int(sp.shape[0]), int(num_heads), int(q_len), None, 0,
              ctypes.addressof(n)))
    items = np.zeros(int(n.value), dtype=np.int32)
    _check(fn(sp.ctypes.data, int(sp.shape[0]), int(num_heads), int(q_len), items.ctypes.data,
              int(items.shape[0]), ctypes.addressof(n)))
    return items


def mla_decode_plan_items_bf16(splits, num_heads: int, q_len: int) -> np.ndarray:
    """The CTA item list for the BF16 entry points."""
    return mla_decode_plan_items(splits, num_heads, q_len, bf16=True)


def mla_decode_workspace_size(batch: int, q_len: int, num_heads: int, max_splits: int) -> int:
    return int(load_library().mla_decode_workspace_size(batch, q_len, num_heads, max_splits))


def mla_decode(q_fp8, kv_pages_fp8, num_pages: int, page_table, max_pages_per_req: int,
               kv_lens, splits, chunks, max_splits: int, kv_split: int, batch: int, q_len: int,
               num_heads: int, causal: bool, q_scale: float, kv_scale: float,
               softmax_scale: float, workspace, workspace_bytes: int, out_bf16, lse_f32=None,
               out_f32_debug=None, stream=None) -> None:
    """Enqueue one decode (split-KV kernel + merge) on `stream`; see mla_decode.h."""
    _decode_call("mla_decode", q_fp8, kv_pages_fp8, num_pages, page_table, max_pages_per_req,
                 kv_lens, splits, chunks, max_splits, kv_split, batch, q_len, num_heads, causal,
                 q_scale, kv_scale, softmax_scale, workspace, workspace_bytes, out_bf16, lse_f32,
                 out_f32_debug, stream)


def _decode_call(fn_name, q_fp8, kv_pages_fp8, num_pages, page_table, max_pages_per_req, kv_lens,
                 splits, chunks, max_splits, kv_split, batch, q_len, num_heads, causal, q_scale,
                 kv_scale, softmax_scale, workspace, workspace_bytes, out_bf16, lse_f32,
                 out_f32_debug, stream):
    fn = getattr(load_library(), fn_name)
    _check(fn(_ptr(q_fp8), _ptr(kv_pages_fp8), int(num_pages), _ptr(page_table),
              int(max_pages_per_req), _ptr(kv_lens), _ptr(splits), _ptr(chunks), int(max_splits),
              int(kv_split), int(batch), int(q_len), int(num_heads), 1 if causal else 0,
              float(q_scale), float(kv_scale), float(softmax_scale), _ptr(workspace),
              int(workspace_bytes), _ptr(out_bf16), _ptr(lse_f32), _ptr(out_f32_debug),
              _stream_handle(stream)))


def mla_decode_ex(q_fp8, kv_pages_fp8, num_pages, page_table, max_pages_per_req, kv_lens, splits,
                  chunks, max_splits, kv_split, batch, q_len, num_heads, causal, q_scale,
                  kv_scale, softmax_scale, workspace, workspace_bytes, out_bf16, lse_f32=None,
                  out_f32_debug=None, *, q_scale_dev=None, kv_scale_dev=None,
                  softmax_scale_dev=None, output_scale: float = 1.0, sinks=None,
                  query_lens=None, kv_bounds=None, cta_items=None, persistent_ctas: int = 0,
                  phases: int = PHASE_ALL, stream=None) -> None:
    """mla_decode with device-side scales, an output scale, attention sinks,
    ragged query counts, key windows and a CTA item list (a device int32
    tensor from mla_decode_plan_items), optionally run by persistent_ctas
    CTAs that loop over the list; phases selects the split-KV kernel or the
    merge alone."""
    opts = DecodeOptions(_ptr(q_scale_dev), _ptr(kv_scale_dev), _ptr(softmax_scale_dev),
                         float(output_scale), _ptr(sinks), _ptr(query_lens), _ptr(kv_bounds),
                         _ptr(cta_items), 0 if cta_items is None else int(cta_items.numel()),
                         int(persistent_ctas), int(phases))
    lib = load_library()
    _check(lib.mla_decode_ex(_ptr(q_fp8), _ptr(kv_pages_fp8), int(num_pages), _ptr(page_table),
                             int(max_pages_per_req), _ptr(kv_lens), _ptr(splits), _ptr(chunks),
                             int(max_splits), int(kv_split), int(batch), int(q_len),
                             int(num_heads), 1 if causal else 0, float(q_scale), float(kv_scale),
                             float(softmax_scale), _ptr(workspace), int(workspace_bytes),
                             _ptr(out_bf16), _ptr(lse_f32), _ptr(out_f32_debug),
                             ctypes.byref(opts), _stream_handle(stream)))


def mla_decode_bf16(q_bf16, kv_pages_bf16, num_pages: int, page_table, max_pages_per_req: int,
                    kv_lens, splits, chunks, max_splits: int, kv_split: int, batch: int,
                    q_len: int, num_heads: int, causal: bool, softmax_scale: float, workspace,
                    workspace_bytes: int, out_bf16, lse_f32=None, out_f32_debug=None,
                    stream=None) -> None:
    """Enqueue one BF16-KV decode (split-KV kernel + merge) on `stream`."""
    lib = load_library()
    _check(lib.mla_decode_bf16(_ptr(q_bf16), _ptr(kv_pages_bf16), int(num_pages),
                               _ptr(page_table), int(max_pages_per_req), _ptr(kv_lens),
                               _ptr(splits), _ptr(chunks), int(max_splits), int(kv_split),
                               int(batch), int(q_len), int(num_heads), 1 if causal else 0,
                               float(softmax_scale), _ptr(workspace), int(workspace_bytes),
                               _ptr(out_bf16), _ptr(lse_f32), _ptr(out_f32_debug),
                               _stream_handle(stream)))


def mla_decode_bf16_ex(q_bf16, kv_pages_bf16, num_pages, page_table, max_pages_per_req, kv_lens,
                       splits, chunks, max_splits, kv_split, batch, q_len, num_heads, causal,
                       softmax_scale, workspace, workspace_bytes, out_bf16, lse_f32=None,
                       out_f32_debug=None, *, softmax_scale_dev=None, output_scale: float = 1.0,
                       sinks=None, query_lens=None, kv_bounds=None, cta_items=None,
                       phases: int = PHASE_ALL, stream=None) -> None:
    """mla_decode_bf16 with a device softmax scale, output scale, sinks,
    ragged query counts, key windows and a CTA item list (a device int32
    tensor from mla_decode_plan_items_bf16); phases as for mla_decode_ex."""
    opts = DecodeOptions(None, None, _ptr(softmax_scale_dev), float(output_scale), _ptr(sinks),
                         _ptr(query_lens), _ptr(kv_bounds), _ptr(cta_items),
                         0 if cta_items is None else int(cta_items.numel()), 0, int(phases))
    lib = load_library()
    _check(lib.mla_decode_bf16_ex(_ptr(q_bf16), _ptr(kv_pages_bf16), int(num_pages),
                                  _ptr(page_table), int(max_pages_per_req), _ptr(kv_lens),
                                  _ptr(splits), _ptr(chunks), int(max_splits), int(kv_split),
                                  int(batch), int(q_len), int(num_heads), 1 if causal else 0,
                                  float(softmax_scale), _ptr(workspace), int(workspace_bytes),
                                  _ptr(out_bf16), _ptr(lse_f32), _ptr(out_f32_debug),
                                  ctypes.byref(opts), _stream_handle(stream)))


def mla_decode_bf16_sparse(q_bf16, kv_pages_bf16, num_pages, page_table, max_pages_per_req,
                           kv_lens, block_idx, topk, splits, chunks, max_splits, kv_split, batch,
                           q_len, num_heads, causal, softmax_scale, workspace, workspace_bytes,
                           out_bf16, lse_f32=None, out_f32_debug=None, *, softmax_scale_dev=None,
                           output_scale: float = 1.0, sinks=None, query_lens=None,
                           kv_bounds=None, cta_items=None, phases: int = PHASE_ALL,
                           stream=None) -> None:
    """BF16 sparse decode over the selected pages block_idx [batch, topk]
    (plan with the compact lengths 32 * topk)."""
    opts = DecodeOptions(None, None, _ptr(softmax_scale_dev), float(output_scale), _ptr(sinks),
                         _ptr(query_lens), _ptr(kv_bounds), _ptr(cta_items),
                         0 if cta_items is None else int(cta_items.numel()), 0, int(phases))
    lib = load_library()
    _check(lib.mla_decode_bf16_sparse(_ptr(q_bf16), _ptr(kv_pages_bf16), int(num_pages),
                                      _ptr(page_table), int(max_pages_per_req), _ptr(kv_lens),
                                      _ptr(block_idx), int(topk), _ptr(splits), _ptr(chunks),
                                      int(max_splits), int(kv_split), int(batch), int(q_len),
                                      int(num_heads), 1 if causal else 0, float(softmax_scale),
                                      _ptr(workspace), int(workspace_bytes), _ptr(out_bf16),
                                      _ptr(lse_f32), _ptr(out_f32_debug), ctypes.byref(opts),
                                      _stream_handle(stream)))


def mla_decode_sparse(q_fp8, kv_pages_fp8, num_pages, page_table, max_pages_per_req, kv_lens,
                      block_idx, topk, splits, chunks, max_splits, kv_split, batch, q_len,
                      num_heads, causal, q_scale, kv_scale, softmax_scale, workspace,
                      workspace_bytes, out_bf16, lse_f32=None, out_f32_debug=None, *,
                      q_scale_dev=None, kv_scale_dev=None, softmax_scale_dev=None,
                      output_scale: float = 1.0, sinks=None, query_lens=None, kv_bounds=None,
                      cta_items=None, persistent_ctas: int = 0, phases: int = PHASE_ALL,
                      stream=None) -> None:
    """Sparse decode over the selected pages block_idx [batch, topk] (plan with
    the compact lengths 32 * topk)."""
    opts = DecodeOptions(_ptr(q_scale_dev), _ptr(kv_scale_dev), _ptr(softmax_scale_dev),
                         float(output_scale), _ptr(sinks), _ptr(query_lens), _ptr(kv_bounds),
                         _ptr(cta_items), 0 if cta_items is None else int(cta_items.numel()),
                         int(persistent_ctas), int(phases))
    lib = load_library()
    _check(lib.mla_decode_sparse(_ptr(q_fp8), _ptr(kv_pages_fp8), int(num_pages),
                                 _ptr(page_table), int(max_pages_per_req), _ptr(kv_lens),
                                 _ptr(block_idx), int(topk), _ptr(splits), _ptr(chunks),
                                 int(max_splits), int(kv_split), int(batch), int(q_len),
                                 int(num_heads), 1 if causal else 0, float(q_scale),
                                 float(kv_scale), float(softmax_scale), _ptr(workspace),
                                 int(workspace_bytes), _ptr(out_bf16), _ptr(lse_f32),
                                 _ptr(out_f32_debug), ctypes.byref(opts),
                                 _stream_handle(stream)))


def _fp4_options(q_scale_dev, kv_scale_dev, softmax_scale_dev, output_scale, sinks, query_lens,
                 kv_bounds, cta_items, phases):
    """The options structure, or None where every option is off."""
    if (q_scale_dev is None and kv_scale_dev is None and softmax_scale_dev is None
            and output_scale == 1.0 and sinks is None and query_lens is None
            and kv_bounds is None and cta_items is None and phases == PHASE_ALL):
        return None
    return ctypes.byref(DecodeOptions(
        _ptr(q_scale_dev), _ptr(kv_scale_dev), _ptr(softmax_scale_dev), float(output_scale),
        _ptr(sinks), _ptr(query_lens), _ptr(kv_bounds), _ptr(cta_items),
        0 if cta_items is None else int(cta_items.numel()), 0, int(phases)))


def _is_fp4_pool(pool) -> bool:
    import torch
    return pool.dtype is torch.uint8 and tuple(pool.shape[1:]) == (FP4_PAGE_BYTES,)


def _fp4_pages(pool, num_pages: int, device: int) -> int:
    if not _is_fp4_pool(pool):
        raise ValueError(f"a 4-bit page pool is uint8 [pages, {FP4_PAGE_BYTES}]")
    return _device_pool(pool, "kv_pages_fp4", device, num_pages, CACHE_FP4)


def mla_decode_fp4(q_fp8, kv_pages_fp4, num_pages, page_table, max_pages_per_req, kv_lens, splits,
                   chunks, max_splits, kv_split, batch, q_len, num_heads, causal, q_scale,
                   kv_scale, softmax_scale, workspace, workspace_bytes, out_bf16, lse_f32=None,
                   out_f32_debug=None, *, q_scale_dev=None, kv_scale_dev=None,
                   softmax_scale_dev=None, output_scale: float = 1.0, sinks=None,
                   query_lens=None, kv_bounds=None, cta_items=None, phases: int = PHASE_ALL,
                   stream=None) -> None:
    """Decode over a 4-bit cache, uint8 [pages, FP4_PAGE_BYTES]; options as for
    mla_decode_ex (no persistent CTAs)."""
    opts = _fp4_options(q_scale_dev, kv_scale_dev, softmax_scale_dev, output_scale, sinks,
                        query_lens, kv_bounds, cta_items, phases)
    dev = _device_of(q_fp8, "q_fp8")
    _call_on(dev, load_library().mla_decode_fp4, _ptr(q_fp8),
             _fp4_pages(kv_pages_fp4, num_pages, dev), num_pages, _ptr(page_table),
             max_pages_per_req, _ptr(kv_lens), _ptr(splits), _ptr(chunks), max_splits, kv_split,
             batch, q_len, num_heads, 1 if causal else 0, q_scale, kv_scale, softmax_scale,
             _ptr(workspace), workspace_bytes, _ptr(out_bf16), _ptr(lse_f32), _ptr(out_f32_debug),
             opts, stream=stream)


def mla_decode_fp4_sparse(q_fp8, kv_pages_fp4, num_pages, page_table, max_pages_per_req, kv_lens,
                          block_idx, topk, splits, chunks, max_splits, kv_split, batch, q_len,
                          num_heads, causal, q_scale, kv_scale, softmax_scale, workspace,
                          workspace_bytes, out_bf16, lse_f32=None, out_f32_debug=None, *,
                          q_scale_dev=None, kv_scale_dev=None, softmax_scale_dev=None,
                          output_scale: float = 1.0, sinks=None, query_lens=None, kv_bounds=None,
                          cta_items=None, phases: int = PHASE_ALL, stream=None) -> None:
    """Sparse decode over the selected pages block_idx [batch, topk] of a 4-bit
    cache (plan with the compact lengths 32 * topk)."""
    opts = _fp4_options(q_scale_dev, kv_scale_dev, softmax_scale_dev, output_scale, sinks,
                        query_lens, kv_bounds, cta_items, phases)
    dev = _device_of(q_fp8, "q_fp8")
    _call_on(dev, load_library().mla_decode_fp4_sparse, _ptr(q_fp8),
             _fp4_pages(kv_pages_fp4, num_pages, dev), num_pages, _ptr(page_table),
             max_pages_per_req, _ptr(kv_lens), _ptr(block_idx), topk, _ptr(splits), _ptr(chunks),
             max_splits, kv_split, batch, q_len, num_heads, 1 if causal else 0, q_scale,
             kv_scale, softmax_scale, _ptr(workspace), workspace_bytes, _ptr(out_bf16),
             _ptr(lse_f32), _ptr(out_f32_debug), opts, stream=stream)


def mla_decode_splitkv(*args, **kw) -> None:
    """Split-KV phase of mla_decode (same arguments)."""
    _decode_call("mla_decode_splitkv", *args, **kw)


def mla_decode_merge(*args, **kw) -> None:
    """Merge phase of mla_decode (same arguments)."""
    _decode_call("mla_decode_merge", *args, **kw)


def mla_decode_workspace_init(workspace, workspace_bytes: int, stream=None) -> None:
    _check(load_library().mla_decode_workspace_init(_ptr(workspace), int(workspace_bytes),
                                                    _stream_handle(stream)))


def mla_merge(partial_o, partial_ml, rows: int, num_ctas_kv: int, kv_split: int, out_bf16,
              lse_f32=None, out_f32_debug=None, stream=None) -> None:
    lib = load_library()
    _check(lib.mla_merge(_ptr(partial_o), _ptr(partial_ml), int(rows), int(num_ctas_kv),
                         int(kv_split), _ptr(out_bf16), _ptr(lse_f32), _ptr(out_f32_debug),
                         _stream_handle(stream)))


def mla_decode_static_ws(q_fp8, kv_pages_fp8, num_pages: int, page_table,
                         max_pages_per_req: int, kv_lens, splits, chunks, max_splits: int,
                         kv_split: int, batch: int, q_len: int, num_heads: int, causal: bool,
                         q_scale: float, kv_scale: float, softmax_scale: float, out_bf16,
                         lse_f32=None, out_f32_debug=None, stream=None) -> None:
    """mla_decode for callers that cannot allocate device memory.

    The scratch lives in a fixed array inside the library
    (MLA_STATIC_WS_BYTES = 16 MiB per GPU), so no workspace is passed.  The
    first call on a device resolves that array's address and should come
    before any stream capture; calls that overlap on the GPU race on the array.
    Device-detected conditions are read with mla_decode_static_ws_status().
    """
    lib = load_library()
    _check(lib.mla_decode_static_ws(
        _ptr(q_fp8), _ptr(kv_pages_fp8), int(num_pages), _ptr(page_table), int(max_pages_per_req),
        _ptr(kv_lens), _ptr(splits), _ptr(chunks), int(max_splits), int(kv_split), int(batch),
        int(q_len), int(num_heads), 1 if causal else 0, float(q_scale), float(kv_scale),
        float(softmax_scale), _ptr(out_bf16), _ptr(lse_f32), _ptr(out_f32_debug),
        _stream_handle(stream)))


STATIC_WS_BYTES = 16 * 1024 * 1024


def mla_decode_static_ws_status(stream=None) -> int:
    """Read and clear the status word of mla_decode_static_ws's fixed scratch
    array (after `stream` drains); raises MlaError on a non-OK status."""
    st = load_library().mla_decode_static_ws_status(_stream_handle(stream))
    _check(st)
    return st


def mla_kv_append(rows_bf16, n_tokens: int, req_idx, positions, page_table,
                  max_pages_per_req: int, batch: int, kv_pages_fp8, num_pages: int,
                  kv_scale: float, status=None, stream=None) -> None:
    """Quantize BF16 latent rows to E4M3 and scatter them into the paged cache."""
    _check(load_library().mla_kv_append(
        _ptr(rows_bf16), int(n_tokens), _ptr(req_idx), _ptr(positions), _ptr(page_table),
        int(max_pages_per_req), int(batch), _ptr(kv_pages_fp8), int(num_pages), float(kv_scale),
        _ptr(status), _stream_handle(stream)))


def _device_of(t, name: str) -> int:
    """Index of the CUDA device that a call's tensors are on: its first one's."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _device_tensor(t, name: str, device: int, dtype=None, least: int = 0, contiguous: bool = True):
    """Address of a tensor on CUDA device `device` (None for None), after the
    checks that a raw address cannot carry: its device, type, contiguity and
    number of elements."""
    if t is None:
        return None
    if t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA tensor on device {device}, like the call's others")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < least:
        raise ValueError(f"{name} has {t.numel()} elements, this call needs {least}")
    return t.data_ptr()


_PAGE_BYTES = {CACHE_FP8: PAGE_SIZE * HEAD_DIM, CACHE_BF16: 2 * PAGE_SIZE * HEAD_DIM,
               CACHE_FP4: FP4_PAGE_BYTES}


def _device_pool(pool, name: str, device: int, pages: int, kind: int):
    """Address of a page pool that holds at least `pages` pages of its kind (an
    unknown kind is left to the library to refuse)."""
    if pool is None:
        return None
    ptr = _device_tensor(pool, name, device)
    if pool.numel() * pool.element_size() < pages * _PAGE_BYTES.get(kind, 0):
        raise ValueError(f"{name} is smaller than {pages} pages of its kind")
    return ptr


def _call_on(index: int, fn, *args, stream=None) -> None:
    """fn(*args, stream) with CUDA device `index` current: on `stream`, or on that
    device's current stream."""
    import torch
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    else:
        handle = _stream_handle(stream)
    if index == torch._C._cuda_getDevice():
        _check(fn(*args, handle))
    else:
        with torch.cuda.device(index):
            _check(fn(*args, handle))


def _row_stride(t, dim: int, name: str) -> int:
    """Stride of a dimension, which the C structure's 0 (contiguous) cannot carry."""
    stride = t.stride(dim)
    if stride == 0:
        raise ValueError(f"{name} may not repeat one row (stride 0)")
    return stride


def mla_prologue(n_tokens: int, *, positions=None, cos_sin=None, rope_positions=None,
                 rope_rows: Optional[int] = None, rope_halves: bool = False, kv_rows=None,
                 norm_weight=None, norm_eps: float = 1e-6, req_idx=None, page_table=None,
                 max_pages_per_req: int = 0, batch: int = 0, kv_pages=None, num_pages: int = 0,
                 cache_kind: int = CACHE_FP8, kv_scale: float = 1.0, q_rows=None,
                 num_heads: int = 0, q_out=None, q_kind: int = CACHE_FP8, q_scale: float = 1.0,
                 status=None, stream=None) -> None:
    """Norm, rotate, quantise and scatter new key rows and rotate and quantise
    the queries, in one launch (see mla_prologue in mla_decode.h).

    kv_rows BF16 [n_tokens, 576] and q_rows BF16 [n_tokens, num_heads, 576] may
    be strided views whose last dimension is dense; either may be None.
    cos_sin is fp32 [rope_rows, 64] (32 cosines, then 32 sines)."""
    import torch
    i32, f32, bf16 = torch.int32, torch.float32, torch.bfloat16
    where = kv_rows if kv_rows is not None else q_rows
    if where is None:
        raise ValueError("mla_prologue needs kv_rows, q_rows or both")
    dev = _device_of(where, "kv_rows" if kv_rows is not None else "q_rows")
    rows = table = pages = weight = None
    row_stride = token_stride = head_stride = 0
    if kv_rows is not None:
        rows = _device_tensor(kv_rows, "kv_rows", dev, bf16, 0, False)
        if kv_rows.dim() != 2 or kv_rows.shape[1] != HEAD_DIM or kv_rows.stride(1) != 1:
            raise ValueError("kv_rows must be [n_tokens, 576] with dense rows")
        if kv_rows.shape[0] < n_tokens:
            raise ValueError("kv_rows has fewer than n_tokens rows")
        if kv_rows.shape[0] > 1:
            row_stride = _row_stride(kv_rows, 0, "kv_rows")
        weight = _device_tensor(norm_weight, "norm_weight", dev, f32, LATENT_DIM)
        table = _device_tensor(page_table, "page_table", dev, i32, batch * max_pages_per_req)
        pages = _device_pool(kv_pages, "kv_pages", dev, num_pages, cache_kind)
    queries = out = None
    if q_rows is not None:
        queries = _device_tensor(q_rows, "q_rows", dev, bf16, 0, False)
        if q_rows.dim() != 3 or q_rows.shape[2] != HEAD_DIM or q_rows.stride(2) != 1:
            raise ValueError("q_rows must be [n_tokens, num_heads, 576] with dense rows")
        if q_rows.shape[0] < n_tokens or q_rows.shape[1] < num_heads:
            raise ValueError("q_rows has fewer than n_tokens tokens or num_heads heads")
        if q_rows.shape[0] > 1:
            token_stride = _row_stride(q_rows, 0, "q_rows")
        if q_rows.shape[1] > 1:
            head_stride = _row_stride(q_rows, 1, "q_rows")
        out = _device_tensor(q_out, "q_out", dev, None, n_tokens * num_heads * HEAD_DIM)
        if out is not None and q_out.element_size() != (2 if q_kind == CACHE_BF16 else 1):
            raise ValueError("q_out must have the element size of q_kind")
    if cos_sin is None:
        rope_rows = 0
    elif rope_rows is None:
        rope_rows = cos_sin.shape[0]
    a = PrologueArgs(n_tokens, _device_tensor(positions, "positions", dev, i32, n_tokens),
                     _device_tensor(cos_sin, "cos_sin", dev, f32, rope_rows * ROPE_DIM),
                     _device_tensor(rope_positions, "rope_positions", dev, i32, n_tokens), rope_rows,
                     1 if rope_halves else 0, rows, row_stride, weight, norm_eps,
                     max_pages_per_req, _device_tensor(req_idx, "req_idx", dev, i32, n_tokens), table,
                     pages,
                     num_pages, batch, cache_kind, kv_scale, q_scale, queries, token_stride,
                     head_stride, out, num_heads, q_kind, _device_tensor(status, "status", dev, i32))
    _call_on(dev, load_library().mla_prologue, ctypes.byref(a), stream=stream)


def mla_pages_copy(src_pool, src_pages: int, src_kind: int, dst_pool, dst_pages: int,
                   dst_kind: int, src_ids, dst_ids, n: int, rows=None, status=None,
                   stream=None) -> None:
    """Copy (or convert, between FP8 and FP4 pools) the first rows[i] rows of
    page src_ids[i] to page dst_ids[i], i < n; ids and rows are int32 CUDA
    tensors."""
    import torch
    i32 = torch.int32
    dev = _device_of(dst_pool, "dst_pool")
    _call_on(dev, load_library().mla_pages_copy,
             _device_pool(src_pool, "src_pool", dev, src_pages, src_kind), src_pages, src_kind,
             _device_pool(dst_pool, "dst_pool", dev, dst_pages, dst_kind), dst_pages, dst_kind,
             _device_tensor(src_ids, "src_ids", dev, i32, n), _device_tensor(dst_ids, "dst_ids", dev, i32, n),
             _device_tensor(rows, "rows", dev, i32, n), n, _device_tensor(status, "status", dev, i32),
             stream=stream)


def mla_pages_remap(page_table, n_entries: int, page_map, num_pages: int, status=None,
                    stream=None) -> None:
    """Replace every page id p >= 0 of a page table by page_map[p], in place."""
    import torch
    i32 = torch.int32
    dev = _device_of(page_table, "page_table")
    _call_on(dev, load_library().mla_pages_remap,
             _device_tensor(page_table, "page_table", dev, i32, n_entries), n_entries,
             _device_tensor(page_map, "page_map", dev, i32, num_pages), num_pages,
             _device_tensor(status, "status", dev, i32), stream=stream)


def _host_ids(ids, name: str) -> np.ndarray:
    """A host list of page ids or counts as int32; ValueError where that would
    change a value."""
    a = np.asarray(ids).reshape(-1)
    if a.size and a.dtype.kind not in "iu":
        raise ValueError(f"{name} must be integers, got {a.dtype}")
    if a.size and (int(a.min()) < -(1 << 31) or int(a.max()) >= 1 << 31):
        raise ValueError(f"{name} does not fit in 32 bits")
    return np.ascontiguousarray(a, dtype=np.int32)


def _host_int(value, name: str, bits: int) -> int:
    """A host integer that the library takes in `bits` bits; ValueError where that
    would change it."""
    try:
        n = operator.index(value)
    except TypeError:
        raise ValueError(f"{name} must be an integer, got {value!r}") from None
    if not -(1 << (bits - 1)) <= n < 1 << (bits - 1):
        raise ValueError(f"{name} does not fit in {bits} bits")
    return n


class PagePool:
    """Reference-counted pages of one cache (mla_pool_*): which are free, forks
    and compactions.  Host only; page ids are int32 numpy arrays.  The copies
    that fork and compact plan run with copy_pages."""

    def __init__(self, num_pages: int):
        self._lib = load_library()
        self.num_pages = _host_int(int(num_pages), "num_pages", 64)
        handle = ctypes.c_void_p()
        _check(self._lib.mla_pool_create(self.num_pages, ctypes.byref(handle)))
        self._handle = handle

    def __reduce__(self):
        raise TypeError("a PagePool cannot be copied or pickled")

    def __del__(self):
        if getattr(self, "_handle", None):
            self._lib.mla_pool_destroy(self._handle)
            self._handle = None

    @property
    def free_pages(self) -> int:
        return int(self._lib.mla_pool_free_pages(self._handle))

    def references(self, page: int) -> int:
        return int(self._lib.mla_pool_references(self._handle, _host_int(page, "page", 32)))

    def alloc(self, n: int) -> np.ndarray:
        """The n lowest free pages; MlaError (MLA_ERR_NO_PAGES) if fewer are free."""
        ids = np.zeros(max(0, int(n)), dtype=np.int32)
        _check(self._lib.mla_pool_alloc(self._handle, int(n), ids.ctypes.data))
        return ids

    def release(self, ids) -> None:
        """Give back one reference of each listed page."""
        ids = _host_ids(ids, "ids")
        _check(self._lib.mla_pool_release(self._handle, ids.ctypes.data, ids.shape[0]))

    def fork(self, ids, kv_len: int, n_forks: int):
        """Fork a request of kv_len tokens: (page lists [n_forks, pages], src,
        dst, rows), the last three the copies to make."""
        ids = _host_ids(ids, "ids")
        pages = (int(kv_len) + PAGE_SIZE - 1) // PAGE_SIZE
        if ids.shape[0] < pages:
            raise ValueError(f"kv_len {kv_len} needs {pages} pages, got {ids.shape[0]}")
        forks = max(0, int(n_forks))
        out = np.zeros((forks, max(0, pages)), dtype=np.int32)
        src, dst, rows = (np.zeros(forks, dtype=np.int32) for _ in range(3))
        n = ctypes.c_int64(0)
        _check(self._lib.mla_pool_fork(self._handle, ids.ctypes.data, int(kv_len), int(n_forks),
                                       out.ctypes.data, src.ctypes.data, dst.ctypes.data,
                                       rows.ctypes.data, ctypes.addressof(n)))
        k = int(n.value)
        return out, src[:k], dst[:k], rows[:k]

    def compact(self, max_moves: Optional[int] = None):
        """Move the pages in use to the low end: (src, dst, map), the copies to
        make and each page's new id."""
        cap = self.num_pages if max_moves is None else int(max_moves)
        src, dst = (np.zeros(max(0, cap), dtype=np.int32) for _ in range(2))
        page_map = np.zeros(self.num_pages, dtype=np.int32)
        n = ctypes.c_int64(0)
        _check(self._lib.mla_pool_compact(self._handle, cap, src.ctypes.data, dst.ctypes.data,
                                          page_map.ctypes.data, ctypes.addressof(n)))
        k = int(n.value)
        return src[:k], dst[:k], page_map


def mla_debug_set_wait_limit(cycles: int) -> None:
    """Test hook: limit of the kernel's pipeline waits (0 = default)."""
    load_library().mla_debug_set_wait_limit(int(cycles))


def mla_debug_set_expire(role: int, tile: int = 0) -> None:
    """Test hook: the pipeline wait `role` at tile `tile` of later launches
    reads as expired (role < 0 = off); see mla_decode.h."""
    load_library().mla_debug_set_expire(int(role), int(tile))


def mla_decode_status(workspace, stream=None) -> int:
    """Read and clear the device status word; raises MlaError on a non-OK status."""
    lib = load_library()
    st = lib.mla_decode_status(_ptr(workspace), _stream_handle(stream))
    _check(st)
    return st


# ---------------------------------------------------------------------------
# Convenience wrappers over torch tensors (allocation on the caller's side).
# ---------------------------------------------------------------------------

def decode(q_fp8, kv_pages_fp8, page_table, kv_lens, *, num_heads: int, q_len: int,
           causal: bool, softmax_scale: float, q_scale: float = 1.0, kv_scale: float = 1.0,
           plan: Optional[Plan] = None, sm_count: Optional[int] = None, target_ctas: int = 0,
           kv_split: Optional[int] = None, want_f32: bool = False, stream=None,
           check_status: bool = True, sinks=None, output_scale: float = 1.0,
           device_scales: bool = False, query_lens=None, kv_bounds=None, block_idx=None,
           use_items: Optional[bool] = None, persistent_ctas: int = 0):
    """Plan, allocate outputs and a workspace with torch, and run mla_decode.

    q_fp8 uint8 [B, q, H, 576] and kv_pages_fp8 uint8 [P, 32, 576] (E4M3 codes)
    and page_table int32 [B, max_pages] are CUDA tensors; kv_lens is a host
    sequence.  With torch.bfloat16 q and kv this runs mla_decode_bf16 (no
    q/kv scales there), with a 4-bit pool (uint8 [P, FP4_PAGE_BYTES])
    mla_decode_fp4.  query_lens [B], kv_bounds [B, 2] and block_idx
    [B, topk] (selected pages: mla_decode_sparse / mla_decode_bf16_sparse,
    planned on the compact lengths) restrict the visible keys.  use_items
    (default: when the plan has empty split slots) launches the split kernel
    over the plan's CTA item list; persistent_ctas > 0 (FP8) runs that list
    with that many persistent CTAs.  Returns (out_bf16, lse, out_f32 or None).
    """
    import torch
    dev = q_fp8.device
    lens = np.asarray(kv_lens.cpu() if hasattr(kv_lens, "cpu") else kv_lens, dtype=np.int32)
    batch = int(lens.shape[0])
    topk = 0 if block_idx is None else int(block_idx.shape[1])
    if plan is None:
        if sm_count is None:
            sm_count = torch.cuda.get_device_properties(dev).multi_processor_count
        plan_lens = lens if block_idx is None else np.full_like(lens, PAGE_SIZE * topk)
        plan = mla_decode_plan(plan_lens, num_heads, q_len, sm_count=sm_count,
                               target_ctas=target_ctas)
    ks = plan.kv_split if kv_split is None else int(kv_split)
    lens_d = torch.from_numpy(lens).to(dev)
    splits_d = torch.from_numpy(plan.splits).to(dev)
    chunks_d = torch.from_numpy(plan.chunks).to(dev)
    ws_bytes = mla_decode_workspace_size(batch, q_len, num_heads, plan.max_splits)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    mla_decode_workspace_init(ws, ws_bytes, stream)
    out = torch.empty((batch, q_len, num_heads, LATENT_DIM), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((batch, q_len, num_heads), dtype=torch.float32, device=dev)
    out_f32 = (torch.empty((batch, q_len, num_heads, LATENT_DIM), dtype=torch.float32, device=dev)
               if want_f32 else None)
    common = (q_fp8, kv_pages_fp8, kv_pages_fp8.shape[0], page_table, page_table.shape[1],
              lens_d, splits_d, chunks_d, plan.max_splits, ks, batch, q_len, num_heads, causal)
    restricted = query_lens is not None or kv_bounds is not None or block_idx is not None
    if use_items is None:
        use_items = bool(np.any(plan.splits < plan.max_splits)) or persistent_ctas > 0
    is_bf16 = q_fp8.dtype == torch.bfloat16
    is_fp4 = not is_bf16 and _is_fp4_pool(kv_pages_fp8)
    if is_fp4 and persistent_ctas > 0:
        raise ValueError("the 4-bit cache has no persistent CTAs")
    items_d = None
    if use_items:
        items_d = torch.from_numpy(
            mla_decode_plan_items(plan.splits, num_heads, q_len, bf16=is_bf16)).to(dev)

    def _dev_i32(x):
        return None if x is None else torch.as_tensor(x, dtype=torch.int32).to(dev).contiguous()
    if is_bf16:
        if kv_pages_fp8.dtype != torch.bfloat16 or q_scale != 1.0 or kv_scale != 1.0:
            raise ValueError("BF16 decode takes BF16 q and kv and no q/kv scales")
        if (sinks is None and output_scale == 1.0 and not device_scales and not restricted
                and items_d is None):
            mla_decode_bf16(*common, softmax_scale, ws, ws_bytes, out, lse, out_f32, stream)
        else:
            sm_d = (torch.tensor([softmax_scale], dtype=torch.float32, device=dev)
                    if device_scales else None)
            sk = None if sinks is None else torch.as_tensor(sinks, dtype=torch.float32).to(dev)
            extra = dict(softmax_scale_dev=sm_d, output_scale=output_scale, sinks=sk,
                         query_lens=_dev_i32(query_lens), kv_bounds=_dev_i32(kv_bounds),
                         cta_items=items_d, stream=stream)
            # With a device scale the host value is a placeholder the kernel must ignore.
            sm_h = 99.0 if device_scales else softmax_scale
            bi_d = _dev_i32(block_idx)
            if bi_d is None:
                mla_decode_bf16_ex(*common, sm_h, ws, ws_bytes, out, lse, out_f32, **extra)
            else:
                mla_decode_bf16_sparse(*common[:6], bi_d, topk, *common[6:], sm_h, ws, ws_bytes,
                                       out, lse, out_f32, **extra)
    elif (sinks is None and output_scale == 1.0 and not device_scales and not restricted
          and items_d is None and persistent_ctas == 0 and not is_fp4):
        mla_decode(*common, q_scale, kv_scale, softmax_scale, ws, ws_bytes, out, lse, out_f32,
                   stream)
    else:
        dev_s = None
        if device_scales:
            dev_s = torch.tensor([q_scale, kv_scale, softmax_scale], dtype=torch.float32,
                                 device=dev)
        sk = None if sinks is None else torch.as_tensor(sinks, dtype=torch.float32).to(dev)
        # With device scales the host values are placeholders the kernel must
        # ignore (deliberately wrong, so a kernel that used them would fail).
        host = (99.0,) * 3 if device_scales else (q_scale, kv_scale, softmax_scale)
        ql_d, kb_d, bi_d = _dev_i32(query_lens), _dev_i32(kv_bounds), _dev_i32(block_idx)
        extra = dict(q_scale_dev=None if dev_s is None else dev_s[0:1],
                     kv_scale_dev=None if dev_s is None else dev_s[1:2],
                     softmax_scale_dev=None if dev_s is None else dev_s[2:3],
                     output_scale=output_scale, sinks=sk, query_lens=ql_d, kv_bounds=kb_d,
                     cta_items=items_d, stream=stream)
        if is_fp4:
            if bi_d is None:
                mla_decode_fp4(*common, *host, ws, ws_bytes, out, lse, out_f32, **extra)
            else:
                mla_decode_fp4_sparse(*common[:6], bi_d, topk, *common[6:], *host, ws, ws_bytes,
                                      out, lse, out_f32, **extra)
            if check_status:
                mla_decode_status(ws, stream)
            return out, lse, out_f32
        extra["persistent_ctas"] = persistent_ctas
        if bi_d is None:
            mla_decode_ex(*common, *host, ws, ws_bytes, out, lse, out_f32, **extra)
        else:
            mla_decode_sparse(*common[:6], bi_d, topk, *common[6:], *host, ws, ws_bytes, out,
                              lse, out_f32, **extra)
    if check_status:
        mla_decode_status(ws, stream)
    return out, lse, out_f32


def fp4_pool(num_pages: int, device="cuda"):
    """A zeroed 4-bit page pool, uint8 [num_pages, FP4_PAGE_BYTES] (CACHE_FP4)."""
    import torch
    return torch.zeros((num_pages, FP4_PAGE_BYTES), dtype=torch.uint8, device=device)


def _cache_kind(pool) -> int:
    """The kind of a page pool, from its type and shape."""
    import torch
    if _is_fp4_pool(pool):
        return CACHE_FP4
    if tuple(pool.shape[1:]) == (PAGE_SIZE, HEAD_DIM):
        if pool.dtype in (torch.uint8, torch.float8_e4m3fn):
            return CACHE_FP8
        if pool.dtype is torch.bfloat16:
            return CACHE_BF16
    raise ValueError("a page pool is uint8 [pages, 32, 576] (E4M3), bfloat16 [pages, 32, 576] "
                     "or uint8 [pages, 10752] (4 bits)")


def _pages_clash(src_at: int, src_kind: int, src, dst_at: int, dst_kind: int, dst) -> bool:
    """Whether a page of src, in a pool at address src_at, shares a byte with one
    of dst (distinct ids) in a pool at dst_at: pools may be views of one allocation."""
    src_bytes, dst_bytes = _PAGE_BYTES[src_kind], _PAGE_BYTES[dst_kind]
    if (src_at + (int(src.max()) + 1) * src_bytes <= dst_at
            or dst_at + (int(dst.max()) + 1) * dst_bytes <= src_at):
        return False
    if src_at == dst_at and src_bytes == dst_bytes:
        return np.intersect1d(src, dst).size > 0
    # The destinations, which do not overlap each other, in order, and for each
    # source the first that ends behind its start.
    src_at = src_at + src.astype(np.int64) * src_bytes
    dst_at = np.sort(dst_at + dst.astype(np.int64) * dst_bytes)
    first = np.searchsorted(dst_at + dst_bytes, src_at, side="right")
    reach = first < dst.shape[0]
    return bool((dst_at[first[reach]] < src_at[reach] + src_bytes).any())


def copy_pages(src_pool, dst_pool, src_ids, dst_ids, rows=None, stream=None) -> None:
    """Copy pages (the lists of PagePool.fork or compact, or any host lists)
    within a pool or between pools, converting between E4M3 and 4-bit pools.

    Lists in which a page would be written twice, or both read and written,
    are refused (ValueError): the copies of one call run in no order."""
    import torch
    src, dst = _host_ids(src_ids, "src_ids"), _host_ids(dst_ids, "dst_ids")
    if src.shape != dst.shape:
        raise ValueError("src_ids and dst_ids must have the same length")
    n = int(src.shape[0])
    if n == 0:
        return
    if src.min() < 0 or src.max() >= src_pool.shape[0] or dst.min() < 0 or \
            dst.max() >= dst_pool.shape[0]:
        raise ValueError("page id outside its pool")
    if np.unique(dst).shape[0] != n:
        raise ValueError("a page is the destination of two copies")
    src_kind, dst_kind = _cache_kind(src_pool), _cache_kind(dst_pool)
    if _pages_clash(src_pool.data_ptr(), src_kind, src, dst_pool.data_ptr(), dst_kind, dst):
        raise ValueError("a page is both a source and a destination")
    lists = [src, dst]
    if rows is not None:
        lists.append(np.broadcast_to(_host_ids(rows, "rows"), (n,)))
        if lists[2].min() < 0 or lists[2].max() > PAGE_SIZE:
            raise ValueError("rows must be in 0..32")
    # One upload for the lists, on the stream that the copy runs on (the lists
    # are pageable host memory: the upload has read them when it returns).
    dev = dst_pool.device
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(dev)):
        lists_d = torch.from_numpy(np.stack(lists)).to(dev)
        mla_pages_copy(src_pool, src_pool.shape[0], src_kind, dst_pool, dst_pool.shape[0],
                       dst_kind, lists_d[0], lists_d[1], n,
                       rows=lists_d[2] if rows is not None else None)


def merge(partial_o, partial_ml, kv_split: int, want_f32: bool = True, stream=None):
    """Run mla_merge on CUDA tensors partial_o [rows, S, 512], partial_ml [rows, S, 2]."""
    import torch
    rows, s = int(partial_o.shape[0]), int(partial_o.shape[1])
    out = torch.empty((rows, LATENT_DIM), dtype=torch.bfloat16, device=partial_o.device)
    lse = torch.empty((rows,), dtype=torch.float32, device=partial_o.device)
    out_f32 = (torch.empty((rows, LATENT_DIM), dtype=torch.float32, device=partial_o.device)
               if want_f32 else None)
    mla_merge(partial_o, partial_ml, rows, s, kv_split, out, lse, out_f32, stream)
    return out, lse, out_f32
