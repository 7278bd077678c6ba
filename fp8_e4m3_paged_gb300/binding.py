"""ctypes binding of libfp8kv_attn.so (the C ABI in include/fp8kv_attn.h).

Argument marshalling only: every step of the attention runs in the library's
CUDA kernels.  Importing this module loads the in-tree shared library and
raises ImportError if it has not been built -- there is no fallback.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp8kv_attn.so")

REVISION = 6
OK = 0
EINVAL = -1
EUNSUPPORTED = -2
EWORKSPACE = -3
EVERSION = -4
ECUDA = -5

MODE_DENSE = 0
MODE_SPARSE_PAGE4 = 1

KV_E4M3 = 0
KV_E5M2 = 1
KV_BF16 = 2

KERNEL_AUTO = 0
KERNEL_GENERIC = 1
KERNEL_TC = 2
KERNEL_TC_SMALL = 3

STATUS_BAD_BLOCK = 0x1
STATUS_BAD_LEN = 0x2
STATUS_BAD_ENTRIES = 0x4
STATUS_TIMEOUT = 0x8

TEST_STALL_PIPELINE = 0x1


class Desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "mode", "batch", "q_max", "num_q_heads", "num_kv_heads", "head_dim", "page_size",
        "max_kv_len", "max_blocks", "num_kv_blocks", "num_sms", "num_splits", "kernel", "kv_format",
        "test_flags")]


class Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "revision", "mode", "batch", "q_max", "num_q_heads", "num_kv_heads", "head_dim",
        "page_size", "max_kv_len", "max_blocks", "num_kv_blocks", "group", "rows",
        "num_splits", "tile_tokens", "kernel")] + [
        ("grid", ctypes.c_int32 * 3),
        ("block_threads", ctypes.c_int32), ("smem_bytes", ctypes.c_int32),
        ("row_chunk", ctypes.c_int32), ("num_sms", ctypes.c_int32),
        ("partial_offset", ctypes.c_int64), ("ml_offset", ctypes.c_int64),
        ("workspace_bytes", ctypes.c_int64),
        ("kv_format", ctypes.c_int32),
        ("test_flags", ctypes.c_int32),
        ("min_part", ctypes.c_int32),
        ("reserved", ctypes.c_int32 * 13),
    ]


class Args(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("k_stride_block", ctypes.c_int64), ("k_stride_token", ctypes.c_int64),
        ("k_stride_head", ctypes.c_int64),
        ("v_stride_block", ctypes.c_int64), ("v_stride_token", ctypes.c_int64),
        ("v_stride_head", ctypes.c_int64),
        ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int64),
        ("row_kv_len", ctypes.c_void_p),
        ("entry_tbl", ctypes.c_void_p), ("entry_mask", ctypes.c_void_p),
        ("n_entries", ctypes.c_void_p), ("entry_stride", ctypes.c_int64),
        ("softmax_scale", ctypes.c_float), ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
        ("k_scale_dev", ctypes.c_void_p), ("v_scale_dev", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("entry_mask_hi", ctypes.c_void_p),
        ("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p),
        ("k_new_stride_req", ctypes.c_int64), ("k_new_stride_token", ctypes.c_int64),
        ("k_new_stride_head", ctypes.c_int64),
        ("v_new_stride_req", ctypes.c_int64), ("v_new_stride_token", ctypes.c_int64),
        ("v_new_stride_head", ctypes.c_int64),
        ("n_new", ctypes.c_int32), ("new_dtype", ctypes.c_int32),
    ]


DTYPE_F16 = 0
DTYPE_BF16 = 1
DTYPE_F32 = 2  # cache read outputs only


class CacheWriteArgs(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("num_kv_blocks", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("k_stride_token", ctypes.c_int64), ("k_stride_head", ctypes.c_int64),
        ("v_stride_token", ctypes.c_int64), ("v_stride_head", ctypes.c_int64),
        ("slot_mapping", ctypes.c_void_p),
        ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("kc_stride_block", ctypes.c_int64), ("kc_stride_token", ctypes.c_int64),
        ("kc_stride_head", ctypes.c_int64),
        ("vc_stride_block", ctypes.c_int64), ("vc_stride_token", ctypes.c_int64),
        ("vc_stride_head", ctypes.c_int64),
        ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
        ("k_scale_dev", ctypes.c_void_p), ("v_scale_dev", ctypes.c_void_p),
        ("status", ctypes.c_void_p), ("kv_format", ctypes.c_int32),
    ]


MERGE_MAX_RANKS = 64


class MergeArgs(ctypes.Structure):
    _fields_ = [
        ("num_ranks", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("num_vectors", ctypes.c_int64),
        ("outs", ctypes.c_void_p), ("rank_stride_out", ctypes.c_int64),
        ("lses", ctypes.c_void_p), ("rank_stride_lse", ctypes.c_int64),
        ("out", ctypes.c_void_p), ("out_f32", ctypes.c_void_p), ("lse_out", ctypes.c_void_p),
    ]


class SelectArgs(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("q_max", ctypes.c_int32), ("topk", ctypes.c_int32),
        ("max_blocks", ctypes.c_int32), ("null_block", ctypes.c_int32),
        ("sel", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int64),
        ("entry_tbl", ctypes.c_void_p), ("entry_mask", ctypes.c_void_p), ("entry_stride", ctypes.c_int64),
        ("n_entries", ctypes.c_void_p), ("status", ctypes.c_void_p),
        ("entry_mask_hi", ctypes.c_void_p),
    ]


CHUNK_AUTO = 0
CHUNK_STREAM = 1
CHUNK_TILE = 2


class ChunkDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "total_q", "max_q", "num_q_heads", "num_kv_heads", "head_dim", "page_size", "max_kv_len",
        "max_blocks", "num_kv_blocks", "window", "sinks", "dtype", "kv_format", "num_sms", "num_splits", "kernel")]


class ChunkPlan(ctypes.Structure):
    same = least = None  # sizes that the tensors must have (fp8kv_attn_chunk_plan)
    _fields_ = [(n, ctypes.c_int32) for n in (
        "revision", "batch", "total_q", "max_q", "num_q_heads", "num_kv_heads", "head_dim", "page_size",
        "max_kv_len", "max_blocks", "num_kv_blocks", "window", "sinks", "dtype", "kv_format", "group", "kernel",
        "num_splits", "row_tiles", "num_sms")] + [
        ("partial_offset", ctypes.c_int64), ("ml_offset", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
        ("min_splits", ctypes.c_int32), ("tree", ctypes.c_int32), ("max_part", ctypes.c_int32),
        ("per_head", ctypes.c_int32), ("reserved", ctypes.c_int32 * 4),
    ]


class ChunkArgs(ctypes.Structure):
    same = least = None  # sizes that the tensors have (make_chunk_args; None: filled by hand)
    _fields_ = [
        ("q", ctypes.c_void_p), ("q_stride_token", ctypes.c_int64), ("q_stride_head", ctypes.c_int64),
        ("out", ctypes.c_void_p), ("out_stride_token", ctypes.c_int64), ("out_stride_head", ctypes.c_int64),
        ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("k_stride_block", ctypes.c_int64), ("k_stride_token", ctypes.c_int64), ("k_stride_head", ctypes.c_int64),
        ("v_stride_block", ctypes.c_int64), ("v_stride_token", ctypes.c_int64), ("v_stride_head", ctypes.c_int64),
        ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int64),
        ("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
        ("softmax_scale", ctypes.c_float), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
        ("k_scale_dev", ctypes.c_void_p), ("v_scale_dev", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class TreeArgs(ctypes.Structure):
    _fields_ = [("chunk", ChunkArgs), ("mask", ctypes.c_void_p), ("mask_stride", ctypes.c_int64),
                ("depth", ctypes.c_void_p)]
    same = least = None  # as ChunkArgs; `words`: what a row of the mask has


class CacheReadArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "total", "num_kv_heads", "head_dim", "page_size", "max_blocks", "num_kv_blocks", "dtype",
        "kv_format")] + [
        ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("kc_stride_block", ctypes.c_int64), ("kc_stride_token", ctypes.c_int64),
        ("kc_stride_head", ctypes.c_int64),
        ("vc_stride_block", ctypes.c_int64), ("vc_stride_token", ctypes.c_int64),
        ("vc_stride_head", ctypes.c_int64),
        ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int64),
        ("cu_len", ctypes.c_void_p), ("start", ctypes.c_void_p),
        ("k_out", ctypes.c_void_p), ("v_out", ctypes.c_void_p),
        ("ko_stride_token", ctypes.c_int64), ("ko_stride_head", ctypes.c_int64),
        ("vo_stride_token", ctypes.c_int64), ("vo_stride_head", ctypes.c_int64),
        ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
        ("k_scale_dev", ctypes.c_void_p), ("v_scale_dev", ctypes.c_void_p), ("status", ctypes.c_void_p),
    ]


class CalibrateArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_tokens", "num_kv_heads", "head_dim", "dtype", "kv_format")] + [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("k_stride_token", ctypes.c_int64), ("k_stride_head", ctypes.c_int64),
        ("v_stride_token", ctypes.c_int64), ("v_stride_head", ctypes.c_int64),
        ("slot_mapping", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
    ]


class CacheScorePlan(ctypes.Structure):
    same = least = None  # as ChunkPlan
    _fields_ = [(n, ctypes.c_int32) for n in (
        "revision", "batch", "total_q", "max_q", "num_q_heads", "num_kv_heads", "head_dim", "page_size",
        "max_kv_len", "max_blocks", "num_kv_blocks", "dtype", "kv_format", "group", "kernel", "num_splits",
        "vectors", "row_tiles", "stat_part", "col_part", "row_groups", "per_head", "num_sms")] + [
        ("partial_offset", ctypes.c_int64), ("ml_offset", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
        ("reserved", ctypes.c_int32 * 7),
    ]


class CacheScoreArgs(ctypes.Structure):
    same = least = None  # as ChunkArgs
    _fields_ = [
        ("q", ctypes.c_void_p), ("q_stride_token", ctypes.c_int64), ("q_stride_head", ctypes.c_int64),
        ("k_cache", ctypes.c_void_p),
        ("k_stride_block", ctypes.c_int64), ("k_stride_token", ctypes.c_int64), ("k_stride_head", ctypes.c_int64),
        ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int64),
        ("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
        ("softmax_scale", ctypes.c_float), ("k_scale", ctypes.c_float), ("k_scale_dev", ctypes.c_void_p),
        ("score_in", ctypes.c_void_p),
        ("score_in_stride_req", ctypes.c_int64), ("score_in_stride_head", ctypes.c_int64),
        ("score", ctypes.c_void_p), ("score_stride_req", ctypes.c_int64), ("score_stride_head", ctypes.c_int64),
        ("decay", ctypes.c_float), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class CacheSelectArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "num_kv_heads", "lists", "max_len", "budget", "sinks", "recent")] + [
        ("score", ctypes.c_void_p), ("score_stride_req", ctypes.c_int64), ("score_stride_head", ctypes.c_int64),
        ("kv_len", ctypes.c_void_p),
        ("keep", ctypes.c_void_p), ("keep_stride_req", ctypes.c_int64), ("keep_stride_list", ctypes.c_int64),
        ("n_keep", ctypes.c_void_p), ("status", ctypes.c_void_p),
    ]


class CacheMoveArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "num_kv_heads", "lists", "max_count", "head_dim", "page_size", "max_blocks", "dst_max_blocks",
        "num_kv_blocks", "kv_format")] + [
        ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("kc_stride_block", ctypes.c_int64), ("kc_stride_token", ctypes.c_int64),
        ("kc_stride_head", ctypes.c_int64),
        ("vc_stride_block", ctypes.c_int64), ("vc_stride_token", ctypes.c_int64),
        ("vc_stride_head", ctypes.c_int64),
        ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int64),
        ("dst_table", ctypes.c_void_p), ("dst_table_stride", ctypes.c_int64),
        ("src", ctypes.c_void_p), ("src_stride_req", ctypes.c_int64), ("src_stride_list", ctypes.c_int64),
        ("count", ctypes.c_void_p), ("first", ctypes.c_void_p),
        ("score", ctypes.c_void_p), ("score_out", ctypes.c_void_p),
        ("score_stride_req", ctypes.c_int64), ("score_stride_head", ctypes.c_int64),
        ("score_out_stride_req", ctypes.c_int64), ("score_out_stride_head", ctypes.c_int64),
        ("max_len", ctypes.c_int32), ("status", ctypes.c_void_p),
    ]


if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m fp8_e4m3_paged_gb300.build_lib` "
        "(the CUDA library is required; there is no CPU fallback)")

lib = ctypes.CDLL(LIB_PATH)
lib.fp8kv_attn_version.restype = ctypes.c_int
lib.fp8kv_attn_version.argtypes = []
lib.fp8kv_attn_strerror.restype = ctypes.c_char_p
lib.fp8kv_attn_strerror.argtypes = [ctypes.c_int]
lib.fp8kv_attn_plan.restype = ctypes.c_int
lib.fp8kv_attn_plan.argtypes = [ctypes.POINTER(Desc), ctypes.POINTER(Plan)]
STATIC_SCRATCH_BYTES = 16 << 20

for _n in ("fp8kv_attn_split", "fp8kv_attn_combine", "fp8kv_attn_forward_static"):
    getattr(lib, _n).restype = ctypes.c_int
    getattr(lib, _n).argtypes = [ctypes.POINTER(Plan), ctypes.POINTER(Args), ctypes.c_void_p]


lib.fp8kv_attn_combine_lse.restype = ctypes.c_int
lib.fp8kv_attn_combine_lse.argtypes = [ctypes.POINTER(Plan), ctypes.POINTER(Args), ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_void_p]
lib.fp8kv_attn_merge.restype = ctypes.c_int
lib.fp8kv_attn_merge.argtypes = [ctypes.POINTER(MergeArgs), ctypes.c_void_p]
lib.fp8kv_attn_merge_scale.restype = ctypes.c_int
lib.fp8kv_attn_merge_scale.argtypes = [ctypes.POINTER(MergeArgs), ctypes.c_int32, ctypes.c_void_p]
lib.fp8kv_attn_select_to_entries.restype = ctypes.c_int
lib.fp8kv_attn_select_to_entries.argtypes = [ctypes.POINTER(SelectArgs), ctypes.c_void_p]
lib.fp8kv_attn_cache_write.restype = ctypes.c_int
lib.fp8kv_attn_cache_write.argtypes = [ctypes.POINTER(CacheWriteArgs), ctypes.c_void_p]
lib.fp8kv_attn_chunk_plan.restype = ctypes.c_int
lib.fp8kv_attn_chunk_plan.argtypes = [ctypes.POINTER(ChunkDesc), ctypes.POINTER(ChunkPlan)]
lib.fp8kv_attn_chunk.restype = ctypes.c_int
lib.fp8kv_attn_chunk.argtypes = [ctypes.POINTER(ChunkPlan), ctypes.POINTER(ChunkArgs), ctypes.c_void_p]
lib.fp8kv_attn_tree_plan.restype = ctypes.c_int
lib.fp8kv_attn_tree_plan.argtypes = [ctypes.POINTER(ChunkDesc), ctypes.POINTER(ChunkPlan)]
lib.fp8kv_attn_tree.restype = ctypes.c_int
lib.fp8kv_attn_tree.argtypes = [ctypes.POINTER(ChunkPlan), ctypes.POINTER(TreeArgs), ctypes.c_void_p]
lib.fp8kv_attn_cache_read.restype = ctypes.c_int
lib.fp8kv_attn_cache_read.argtypes = [ctypes.POINTER(CacheReadArgs), ctypes.c_void_p]
lib.fp8kv_attn_cache_score_plan.restype = ctypes.c_int
lib.fp8kv_attn_cache_score_plan.argtypes = [ctypes.POINTER(ChunkDesc), ctypes.POINTER(CacheScorePlan)]
lib.fp8kv_attn_cache_score.restype = ctypes.c_int
lib.fp8kv_attn_cache_score.argtypes = [ctypes.POINTER(CacheScorePlan), ctypes.POINTER(CacheScoreArgs), ctypes.c_void_p]
lib.fp8kv_attn_cache_select.restype = ctypes.c_int
lib.fp8kv_attn_cache_select.argtypes = [ctypes.POINTER(CacheSelectArgs), ctypes.c_void_p]
lib.fp8kv_attn_cache_move.restype = ctypes.c_int
lib.fp8kv_attn_cache_move.argtypes = [ctypes.POINTER(CacheMoveArgs), ctypes.c_void_p]
lib.fp8kv_attn_cache_calibrate.restype = ctypes.c_int
lib.fp8kv_attn_cache_calibrate.argtypes = [ctypes.POINTER(CalibrateArgs), ctypes.c_void_p]


class Fp8kvError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {fp8kv_attn_strerror(code)} ({code})")


def fp8kv_attn_version() -> int:
    return lib.fp8kv_attn_version()


def fp8kv_attn_strerror(code: int) -> str:
    return lib.fp8kv_attn_strerror(code).decode()


def fp8kv_attn_plan(desc: Desc) -> Plan:
    plan = Plan()
    rc = lib.fp8kv_attn_plan(ctypes.byref(desc), ctypes.byref(plan))
    if rc != OK:
        raise Fp8kvError(rc, "fp8kv_attn_plan")
    return plan


def fp8kv_attn_split(plan: Plan, args: Args, stream: int = 0) -> None:
    rc = lib.fp8kv_attn_split(ctypes.byref(plan), ctypes.byref(args), ctypes.c_void_p(stream))
    if rc != OK:
        raise Fp8kvError(rc, "fp8kv_attn_split")


def fp8kv_attn_combine(plan: Plan, args: Args, stream: int = 0) -> None:
    rc = lib.fp8kv_attn_combine(ctypes.byref(plan), ctypes.byref(args), ctypes.c_void_p(stream))
    if rc != OK:
        raise Fp8kvError(rc, "fp8kv_attn_combine")


def fp8kv_attn_forward_static(plan: Plan, args: Args, stream: int = 0) -> None:
    """Split + combine using the library's own device scratch (no workspace)."""
    rc = lib.fp8kv_attn_forward_static(ctypes.byref(plan), ctypes.byref(args), ctypes.c_void_p(stream))
    if rc != OK:
        raise Fp8kvError(rc, "fp8kv_attn_forward_static")


# ---------------------------------------------------------------- torch glue

def make_desc(*, mode: int, batch: int, q_max: int, num_q_heads: int, num_kv_heads: int,
              head_dim: int, page_size: int, max_kv_len: int, max_blocks: int,
              num_kv_blocks: int, num_sms: int = 0, num_splits: int = 0, kernel: int = 0,
              kv_format: int = KV_E4M3, test_flags: int = 0) -> Desc:
    return Desc(mode, batch, q_max, num_q_heads, num_kv_heads, head_dim, page_size,
                max_kv_len, max_blocks, num_kv_blocks, num_sms, num_splits, kernel, kv_format,
                test_flags)


def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def make_args(*, q, k_cache, v_cache, out, workspace, softmax_scale: float,
              k_scale: float = 1.0, v_scale: float = 1.0,
              block_table=None, row_kv_len=None,
              entry_tbl=None, entry_mask=None, n_entries=None,
              k_scale_dev=None, v_scale_dev=None, entry_mask_hi=None, k_new=None, v_new=None) -> Args:
    """Fill an Args struct from torch CUDA tensors.

    k_cache / v_cache: uint8 tensors indexed [block][slot][kv_head][d] (any
    strides with d contiguous); q / out: fp16 [B][q_max][Hq][D] contiguous;
    workspace: a uint8 tensor of at least plan.workspace_bytes bytes.
    k_new / v_new (fused write of a verify step's new tokens): fp16 or bf16
    [B][n_new][Hkv][D], d contiguous.
    """
    a = Args()
    a.q = _ptr(q)
    a.k_cache = _ptr(k_cache)
    a.v_cache = _ptr(v_cache)
    ks = k_cache.stride()
    vs = v_cache.stride()
    eb_k = k_cache.element_size()
    eb_v = v_cache.element_size()
    a.k_stride_block, a.k_stride_token, a.k_stride_head = ks[0] * eb_k, ks[1] * eb_k, ks[2] * eb_k
    a.v_stride_block, a.v_stride_token, a.v_stride_head = vs[0] * eb_v, vs[1] * eb_v, vs[2] * eb_v
    if block_table is not None:
        a.block_table = _ptr(block_table)
        a.block_table_stride = block_table.stride(0)
    a.row_kv_len = _ptr(row_kv_len)
    if entry_tbl is not None:
        a.entry_tbl = _ptr(entry_tbl)
        a.entry_stride = entry_tbl.stride(0)
    a.entry_mask = _ptr(entry_mask)
    a.entry_mask_hi = _ptr(entry_mask_hi)
    a.n_entries = _ptr(n_entries)
    a.softmax_scale = float(softmax_scale)
    a.k_scale = float(k_scale)
    a.v_scale = float(v_scale)
    a.k_scale_dev = _ptr(k_scale_dev)
    a.v_scale_dev = _ptr(v_scale_dev)
    a.out = _ptr(out)
    a.workspace = _ptr(workspace)
    a.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if k_new is not None:
        import torch

        a.k_new, a.v_new = _ptr(k_new), _ptr(v_new)
        a.k_new_stride_req, a.k_new_stride_token, a.k_new_stride_head = k_new.stride()[:3]
        a.v_new_stride_req, a.v_new_stride_token, a.v_new_stride_head = v_new.stride()[:3]
        a.n_new = k_new.shape[1]
        a.new_dtype = DTYPE_F16 if k_new.dtype == torch.float16 else DTYPE_BF16
    return a


@dataclass
class Call:
    """A planned split + combine over fixed device buffers (graph friendly)."""
    plan: Plan
    args: Args

    def split(self, stream: int) -> None:
        fp8kv_attn_split(self.plan, self.args, stream)

    def combine(self, stream: int) -> None:
        fp8kv_attn_combine(self.plan, self.args, stream)

    def run(self, stream: int) -> None:
        self.split(stream)
        self.combine(stream)


def fp8kv_attn_cache_write(args: CacheWriteArgs, stream: int = 0) -> None:
    rc = lib.fp8kv_attn_cache_write(ctypes.byref(args), ctypes.c_void_p(stream))
    if rc != OK:
        raise Fp8kvError(rc, "fp8kv_attn_cache_write")


def make_cache_write_args(*, k, v, slot_mapping, k_cache, v_cache, page_size: int,
                          k_scale: float = 1.0, v_scale: float = 1.0, k_scale_dev=None,
                          v_scale_dev=None, status=None, kv_format: int = KV_E4M3) -> CacheWriteArgs:
    """Fill a CacheWriteArgs struct from torch CUDA tensors.

    k / v: float16 or bfloat16 [N][Hkv][D] (d contiguous); slot_mapping:
    int64 [N]; k_cache / v_cache: uint8 [blocks][page_size][Hkv][D] views
    (d contiguous); status: optional int32 tensor of one element."""
    import torch

    a = CacheWriteArgs()
    N, Hkv, D = k.shape
    a.num_tokens, a.num_kv_heads, a.head_dim = N, Hkv, D
    a.page_size = page_size
    a.num_kv_blocks = k_cache.shape[0]
    a.dtype = DTYPE_F16 if k.dtype == torch.float16 else DTYPE_BF16
    a.k, a.v = _ptr(k), _ptr(v)
    a.k_stride_token, a.k_stride_head = k.stride(0), k.stride(1)
    a.v_stride_token, a.v_stride_head = v.stride(0), v.stride(1)
    a.slot_mapping = _ptr(slot_mapping)
    a.k_cache, a.v_cache = _ptr(k_cache), _ptr(v_cache)
    a.kc_stride_block, a.kc_stride_token, a.kc_stride_head = k_cache.stride()[:3]
    a.vc_stride_block, a.vc_stride_token, a.vc_stride_head = v_cache.stride()[:3]
    a.k_scale, a.v_scale = float(k_scale), float(v_scale)
    a.k_scale_dev, a.v_scale_dev = _ptr(k_scale_dev), _ptr(v_scale_dev)
    a.status = _ptr(status)
    a.kv_format = kv_format
    return a


def fp8kv_attn_combine_lse(plan: Plan, args: Args, out_f32, lse, stream: int = 0) -> None:
    """Combine one rank's shard into FP32 output [B][q][Hq][D] and base-2 LSE [B][q][Hq]."""
    rc = lib.fp8kv_attn_combine_lse(ctypes.byref(plan), ctypes.byref(args), _ptr(out_f32), _ptr(lse),
                                    ctypes.c_void_p(stream))
    if rc != OK:
        raise Fp8kvError(rc, "fp8kv_attn_combine_lse")


def make_merge_args(*, outs, lses, out=None, out_f32=None, lse_out=None) -> MergeArgs:
    """outs: FP32 [R][n..][D]; lses: FP32 [R][n..] (torch CUDA tensors; the
    vector dimensions are flattened, the rank dimension may be strided)."""
    R, D = outs.shape[0], outs.shape[-1]
    a = MergeArgs()
    a.num_ranks, a.head_dim = R, D
    a.num_vectors = lses[0].numel() if R > 0 else 0
    a.outs, a.rank_stride_out = _ptr(outs), outs.stride(0)
    a.lses, a.rank_stride_lse = _ptr(lses), lses.stride(0)
    a.out, a.out_f32, a.lse_out = _ptr(out), _ptr(out_f32), _ptr(lse_out)
    return a


def fp8kv_attn_merge(args: MergeArgs, stream: int = 0) -> None:
    rc = lib.fp8kv_attn_merge(ctypes.byref(args), ctypes.c_void_p(stream))
    if rc != OK:
        raise Fp8kvError(rc, "fp8kv_attn_merge")


def fp8kv_attn_merge_scale(args: MergeArgs, rank: int, stream: int = 0) -> None:
    rc = lib.fp8kv_attn_merge_scale(ctypes.byref(args), rank, ctypes.c_void_p(stream))
    if rc != OK:
        raise Fp8kvError(rc, "fp8kv_attn_merge_scale")


def make_select_args(*, sel, block_table, max_blocks: int, null_block: int, entry_tbl, entry_mask,
                     n_entries, status=None, entry_mask_hi=None) -> SelectArgs:
    """sel: int32 [B][q][topk]; block_table: int32 [B][>= max_blocks];
    entry_tbl / entry_mask (/ entry_mask_hi for q > 8): int32 [B][stride]
    (the mask tensors hold the uint32 bit patterns); n_entries: int32 [B]
    (torch CUDA tensors)."""
    a = SelectArgs()
    a.batch, a.q_max, a.topk = sel.shape
    a.max_blocks, a.null_block = max_blocks, null_block
    a.sel = _ptr(sel)
    a.block_table, a.block_table_stride = _ptr(block_table), block_table.stride(0)
    a.entry_tbl, a.entry_mask, a.entry_stride = _ptr(entry_tbl), _ptr(entry_mask), entry_tbl.stride(0)
    a.n_entries, a.status = _ptr(n_entries), _ptr(status)
    a.entry_mask_hi = _ptr(entry_mask_hi)
    return a


def fp8kv_attn_select_to_entries(args: SelectArgs, stream: int = 0) -> None:
    rc = lib.fp8kv_attn_select_to_entries(ctypes.byref(args), ctypes.c_void_p(stream))
    if rc != OK:
        raise Fp8kvError(rc, "fp8kv_attn_select_to_entries")


# ---------------------------------------------------------------- chunk attention, cache read, calibration

def _torch_dtype(t, *allowed) -> int:
    import torch

    code = {torch.float16: DTYPE_F16, torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}.get(t.dtype, -1)
    if code not in allowed:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return code


def _check(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _one_device(*tensors) -> None:
    """The call's tensors lie on one GPU (pinned host tensors may stand beside them)."""
    on = {t.device for t in tensors if t is not None and t.device.type != "cpu"}
    _check(len(on) <= 1, f"tensors on several devices: {', '.join(sorted(map(str, on)))}")


def _int32(t, n: int, name: str) -> None:
    import torch

    _check(t.dtype == torch.int32 and t.dim() == 1 and t.numel() == n and t.is_contiguous(),
           f"{name}: a contiguous int32 tensor of {n} elements")


def _device_scale(t, name: str) -> None:
    import torch

    _check(t is None or (t.dtype == torch.float32 and t.numel() == 1), f"{name}: one float32 element")


def _pages(t, name: str):
    """Byte strides (block, token, head) of a cache view [blocks][page][Hkv][D], d contiguous."""
    _check(t.dim() == 4 and t.element_size() == 1 and t.stride(3) == 1,
           f"{name}: one-byte elements [blocks][page][Hkv][D] with d contiguous")
    return t.stride()[:3]


def _rows(t, name: str):
    _check(t.dim() == 3 and t.stride(2) == 1, f"{name}: [rows][heads][D] with d contiguous")
    return t.stride()[:2]


def _table(t, name: str):
    """Address and row stride of a block table [B][columns]."""
    import torch

    rows, cols = t.shape if t.dim() == 2 else (-1, -1)
    _check(t.dtype == torch.int32 and rows >= 0 and (t.stride(1) == 1 or cols <= 1),
           f"{name}: int32 [B][columns], columns contiguous")
    if rows <= 1:  # one request: its next row is never read, whatever the stride says
        return _ptr(t), max(t.stride(0), cols)
    _check(t.stride(0) >= cols, f"{name}: rows that overlap (a table that all requests share needs a copy for each)")
    return _ptr(t), t.stride(0)


def make_chunk_desc(*, batch: int, total_q: int, max_q: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                    page_size: int, max_kv_len: int, max_blocks: int, num_kv_blocks: int, window: int = 0,
                    sinks: int = 0, dtype: int = DTYPE_F16, kv_format: int = KV_E4M3, num_sms: int = 0,
                    num_splits: int = 0, kernel: int = CHUNK_AUTO) -> ChunkDesc:
    return ChunkDesc(batch, total_q, max_q, num_q_heads, num_kv_heads, head_dim, page_size, max_kv_len, max_blocks,
                     num_kv_blocks, window, sinks, dtype, kv_format, num_sms, num_splits, kernel)


def fp8kv_attn_chunk_plan(desc: ChunkDesc) -> ChunkPlan:
    return _chunk_plan(lib.fp8kv_attn_chunk_plan, desc, "fp8kv_attn_chunk_plan")


def _chunk_plan(make, desc: ChunkDesc, name: str) -> ChunkPlan:
    plan = ChunkPlan()
    rc = make(ctypes.byref(desc), ctypes.byref(plan))
    if rc != OK:
        raise Fp8kvError(rc, name)
    # what the tensors must have (make_chunk_args notes what they have): the same ..., and at least ...
    plan.same = (plan.num_q_heads, plan.num_kv_heads, plan.head_dim, plan.page_size, plan.dtype)
    plan.least = (plan.batch, plan.total_q, plan.max_blocks, plan.num_kv_blocks)
    return plan


def make_chunk_args(*, q, k_cache, v_cache, out, workspace, softmax_scale: float, block_table, cu_q, kv_len,
                    k_scale: float = 1.0, v_scale: float = 1.0, k_scale_dev=None, v_scale_dev=None) -> ChunkArgs:
    """Fill a ChunkArgs struct from torch CUDA tensors.

    q / out: fp16 or bf16 [total_q][Hq][D] (any row and head strides, d
    contiguous); k_cache / v_cache: uint8 [blocks][page][Hkv][D] views;
    block_table: int32 [B][columns], a row of its own for each request; cu_q:
    int32 [B+1]; kv_len: int32 [B]; workspace: a uint8 tensor of at least
    plan.workspace_bytes bytes, its first four bytes (the status word) zeroed
    once.  fp8kv_attn_chunk compares the tensors with the plan: the same heads,
    head dim, page size and type, and at least its requests, rows, table columns
    and blocks."""
    dtype = _torch_dtype(q, DTYPE_F16, DTYPE_BF16)
    _check(out.dtype == q.dtype and out.shape == q.shape, "out: same type and shape as q")
    table, table_stride = _table(block_table, "block_table")
    _int32(cu_q, block_table.shape[0] + 1, "cu_q")
    _int32(kv_len, block_table.shape[0], "kv_len")
    _device_scale(k_scale_dev, "k_scale_dev")
    _device_scale(v_scale_dev, "v_scale_dev")
    _one_device(q, k_cache, v_cache, out, workspace, block_table, cu_q, kv_len, k_scale_dev, v_scale_dev)
    a = ChunkArgs()
    a.q, (a.q_stride_token, a.q_stride_head) = _ptr(q), _rows(q, "q")
    a.out, (a.out_stride_token, a.out_stride_head) = _ptr(out), _rows(out, "out")
    a.k_cache, a.v_cache = _ptr(k_cache), _ptr(v_cache)
    a.k_stride_block, a.k_stride_token, a.k_stride_head = _pages(k_cache, "k_cache")
    a.v_stride_block, a.v_stride_token, a.v_stride_head = _pages(v_cache, "v_cache")
    a.block_table, a.block_table_stride = table, table_stride
    a.cu_q, a.kv_len = _ptr(cu_q), _ptr(kv_len)
    a.softmax_scale, a.k_scale, a.v_scale = float(softmax_scale), float(k_scale), float(v_scale)
    a.k_scale_dev, a.v_scale_dev = _ptr(k_scale_dev), _ptr(v_scale_dev)
    a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    _check(k_cache.shape[1:] == v_cache.shape[1:], "v_cache: pages of the same shape as k_cache's")
    _check(q.shape[2] == k_cache.shape[3], "q: the caches' head dim")
    a.same = (q.shape[1], *k_cache.shape[2:], k_cache.shape[1], dtype)
    a.least = (block_table.shape[0], q.shape[0], block_table.shape[1], min(k_cache.shape[0], v_cache.shape[0]))
    return a


def _fits(plan, args) -> None:
    """The tensors are those that the plan is for."""
    same = args.same
    if same is not None and plan.same is not None:
        _check(same == plan.same, "the plan's heads, head dim, page size and type are not those of the tensors")
        (b, n, c, k), (pb, pn, pc, pk) = args.least, plan.least
        if b < pb or n < pn or c < pc or k < pk:
            raise ValueError("the plan has more requests, rows, table columns or blocks than the tensors")


def fp8kv_attn_chunk(plan: ChunkPlan, args: ChunkArgs, stream: int = 0) -> None:
    _fits(plan, args)
    rc = lib.fp8kv_attn_chunk(ctypes.byref(plan), ctypes.byref(args), stream)
    if rc != OK:
        raise Fp8kvError(rc, "fp8kv_attn_chunk")


@dataclass
class ChunkCall:
    """A planned chunk attention over fixed device buffers (graph friendly)."""
    plan: ChunkPlan
    args: ChunkArgs

    def run(self, stream: int) -> None:
        fp8kv_attn_chunk(self.plan, self.args, stream)


def fp8kv_attn_tree_plan(desc: ChunkDesc) -> ChunkPlan:
    return _chunk_plan(lib.fp8kv_attn_tree_plan, desc, "fp8kv_attn_tree_plan")


def make_tree_args(*, mask, depth=None, **chunk) -> TreeArgs:
    """Fill a TreeArgs struct from torch CUDA tensors.

    chunk: as for make_chunk_args; mask: int32 [total_q][words] (the uint32 bit
    patterns), words contiguous, at least one for 32 nodes of the plan's max_q;
    depth: int32 [total_q], needed with a window."""
    import torch

    q = chunk["q"]
    _check(mask.dtype == torch.int32 and mask.dim() == 2 and mask.shape[0] == q.shape[0] and
           (mask.stride(1) == 1 or mask.shape[1] <= 1) and mask.stride(0) >= 0,
           "mask: int32 [total_q][words], words contiguous")
    if depth is not None:
        _int32(depth, q.shape[0], "depth")
    _one_device(q, mask, depth)
    a = TreeArgs()
    made = make_chunk_args(**chunk)
    a.chunk = made
    a.mask, a.mask_stride, a.depth = _ptr(mask), mask.stride(0), _ptr(depth)
    if mask.shape[0] <= 1:  # one row: its next is never read
        a.mask_stride = max(mask.stride(0), mask.shape[1])
    a.same, a.least, a.words = made.same, made.least, mask.shape[1]
    return a


def fp8kv_attn_tree(plan: ChunkPlan, args: TreeArgs, stream: int = 0) -> None:
    _fits(plan, args)
    if args.same is not None:
        _check(32 * args.words >= plan.max_q, "mask: fewer words than the plan's max_q nodes take")
    rc = lib.fp8kv_attn_tree(ctypes.byref(plan), ctypes.byref(args), stream)
    if rc != OK:
        raise Fp8kvError(rc, "fp8kv_attn_tree")


@dataclass
class TreeCall:
    """A planned tree attention over fixed device buffers (graph friendly)."""
    plan: ChunkPlan
    args: TreeArgs

    def run(self, stream: int) -> None:
        fp8kv_attn_tree(self.plan, self.args, stream)


def make_cache_read_args(*, k_cache, v_cache, block_table, cu_len, k_out, v_out, start=None, k_scale: float = 1.0,
                         v_scale: float = 1.0, k_scale_dev=None, v_scale_dev=None, status=None,
                         kv_format: int = KV_E4M3) -> CacheReadArgs:
    """Fill a CacheReadArgs struct from torch CUDA tensors.

    k_cache / v_cache: uint8 [blocks][page][Hkv][D] views; block_table: int32
    [B][columns]; cu_len: int32 [B+1]; start: optional int32 [B]; k_out /
    v_out: fp16, bf16 or fp32 [total][Hkv][D] (d contiguous); status: optional
    int32 tensor of one element."""
    _one_device(k_cache, v_cache, block_table, cu_len, k_out, v_out, start, k_scale_dev, v_scale_dev, status)
    a = CacheReadArgs()
    a.dtype = _torch_dtype(k_out, DTYPE_F16, DTYPE_BF16, DTYPE_F32)
    _check(v_out.dtype == k_out.dtype and v_out.shape == k_out.shape, "v_out: same type and shape as k_out")
    _check(k_cache.shape == v_cache.shape and k_out.shape[1:] == k_cache.shape[2:],
           "k_out / v_out: [total][Hkv][D] with the caches' Hkv and D")
    table, table_stride = _table(block_table, "block_table")
    _int32(cu_len, block_table.shape[0] + 1, "cu_len")
    if start is not None:
        _int32(start, block_table.shape[0], "start")
    _device_scale(k_scale_dev, "k_scale_dev")
    _device_scale(v_scale_dev, "v_scale_dev")
    a.batch, a.max_blocks = block_table.shape
    a.total, a.num_kv_heads, a.head_dim = k_out.shape
    a.num_kv_blocks, a.page_size = k_cache.shape[:2]
    a.kv_format = kv_format
    a.k_cache, a.v_cache = _ptr(k_cache), _ptr(v_cache)
    a.kc_stride_block, a.kc_stride_token, a.kc_stride_head = _pages(k_cache, "k_cache")
    a.vc_stride_block, a.vc_stride_token, a.vc_stride_head = _pages(v_cache, "v_cache")
    a.block_table, a.block_table_stride = table, table_stride
    a.cu_len, a.start = _ptr(cu_len), _ptr(start)
    a.k_out, (a.ko_stride_token, a.ko_stride_head) = _ptr(k_out), _rows(k_out, "k_out")
    a.v_out, (a.vo_stride_token, a.vo_stride_head) = _ptr(v_out), _rows(v_out, "v_out")
    a.k_scale, a.v_scale = float(k_scale), float(v_scale)
    a.k_scale_dev, a.v_scale_dev, a.status = _ptr(k_scale_dev), _ptr(v_scale_dev), _ptr(status)
    return a


def fp8kv_attn_cache_read(args: CacheReadArgs, stream: int = 0) -> None:
    rc = lib.fp8kv_attn_cache_read(ctypes.byref(args), stream)
    if rc != OK:
        raise Fp8kvError(rc, "fp8kv_attn_cache_read")


def make_calibrate_args(*, k, v, k_scale, v_scale, slot_mapping=None, kv_format: int = KV_E4M3) -> CalibrateArgs:
    """Fill a CalibrateArgs struct from torch CUDA tensors.

    k / v: fp16 or bf16 [N][Hkv][D] (d contiguous); k_scale / v_scale: float32
    tensors of one element, raised in place; slot_mapping: optional int64 [N]
    (tokens with a negative slot do not count)."""
    import torch

    _one_device(k, v, k_scale, v_scale, slot_mapping)
    a = CalibrateArgs()
    a.dtype = _torch_dtype(k, DTYPE_F16, DTYPE_BF16)
    _check(v.dtype == k.dtype and v.shape == k.shape, "v: same type and shape as k")
    _check(k_scale is not None and v_scale is not None, "k_scale, v_scale: float32 tensors of one element")
    _device_scale(k_scale, "k_scale")
    _device_scale(v_scale, "v_scale")
    if slot_mapping is not None:
        _check(slot_mapping.dtype == torch.int64 and slot_mapping.numel() == k.shape[0] and
               slot_mapping.is_contiguous(), "slot_mapping: a contiguous int64 tensor of N elements")
    a.num_tokens, a.num_kv_heads, a.head_dim = k.shape
    a.kv_format = kv_format
    a.k, (a.k_stride_token, a.k_stride_head) = _ptr(k), _rows(k, "k")
    a.v, (a.v_stride_token, a.v_stride_head) = _ptr(v), _rows(v, "v")
    a.slot_mapping, a.k_scale, a.v_scale = _ptr(slot_mapping), _ptr(k_scale), _ptr(v_scale)
    return a


def fp8kv_attn_cache_calibrate(args: CalibrateArgs, stream: int = 0) -> None:
    rc = lib.fp8kv_attn_cache_calibrate(ctypes.byref(args), stream)
    if rc != OK:
        raise Fp8kvError(rc, "fp8kv_attn_cache_calibrate")


# ---------------------------------------------------------------- which positions stay, and their move

def _status(t) -> None:
    import torch

    _check(t is None or (t.dtype in (torch.int32, torch.uint32) and t.numel() == 1), "status: one int32 element")


def _lists(t, name: str):
    """Strides (request, list) of an int32 tensor [B][lists][entries], entries contiguous."""
    import torch

    _check(t.dtype == torch.int32 and t.dim() == 3 and (t.stride(2) == 1 or t.shape[2] <= 1),
           f"{name}: int32 [B][lists][entries], entries contiguous")
    return t.stride()[:2]


def _weights(t, name: str):
    """Strides (request, head) of a float32 tensor [B][Hkv][positions], positions contiguous."""
    import torch

    _check(t.dtype == torch.float32 and t.dim() == 3 and (t.stride(2) == 1 or t.shape[2] <= 1),
           f"{name}: float32 [B][Hkv][positions], positions contiguous")
    return t.stride()[:2]


def fp8kv_attn_cache_score_plan(desc: ChunkDesc) -> CacheScorePlan:
    plan = CacheScorePlan()
    rc = lib.fp8kv_attn_cache_score_plan(ctypes.byref(desc), ctypes.byref(plan))
    if rc != OK:
        raise Fp8kvError(rc, "fp8kv_attn_cache_score_plan")
    plan.same = (plan.num_q_heads, plan.num_kv_heads, plan.head_dim, plan.page_size, plan.dtype)
    plan.least = (plan.batch, plan.total_q, plan.max_blocks, plan.num_kv_blocks)
    return plan


def make_cache_score_args(*, q, k_cache, block_table, cu_q, kv_len, softmax_scale: float, score, workspace,
                          score_in=None, decay: float = 1.0, k_scale: float = 1.0, k_scale_dev=None) -> CacheScoreArgs:
    """Fill a CacheScoreArgs struct from torch CUDA tensors.

    q, k_cache, block_table, cu_q, kv_len, workspace: as for make_chunk_args;
    score, score_in: float32 [B][Hkv][at least the plan's max_kv_len] (positions
    contiguous), score_in None (nothing gathered before), score itself, or a
    buffer that does not overlap it."""
    dtype = _torch_dtype(q, DTYPE_F16, DTYPE_BF16)
    table, table_stride = _table(block_table, "block_table")
    b = block_table.shape[0]
    _int32(cu_q, b + 1, "cu_q")
    _int32(kv_len, b, "kv_len")
    _device_scale(k_scale_dev, "k_scale_dev")
    _one_device(q, k_cache, block_table, cu_q, kv_len, k_scale_dev, score, score_in, workspace)
    a = CacheScoreArgs()
    a.q, (a.q_stride_token, a.q_stride_head) = _ptr(q), _rows(q, "q")
    a.k_cache = _ptr(k_cache)
    a.k_stride_block, a.k_stride_token, a.k_stride_head = _pages(k_cache, "k_cache")
    a.block_table, a.block_table_stride = table, table_stride
    a.cu_q, a.kv_len = _ptr(cu_q), _ptr(kv_len)
    a.softmax_scale, a.k_scale, a.k_scale_dev = float(softmax_scale), float(k_scale), _ptr(k_scale_dev)
    a.score, (a.score_stride_req, a.score_stride_head) = _ptr(score), _weights(score, "score")
    _check(score.shape[:2] == (b, k_cache.shape[2]), "score: [B][Hkv][positions]")
    if score_in is not None:
        a.score_in, (a.score_in_stride_req, a.score_in_stride_head) = _ptr(score_in), _weights(score_in, "score_in")
        _check(score_in.shape == score.shape, "score_in: the same shape as score")
    a.decay = float(decay)
    a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    _check(q.shape[2] == k_cache.shape[3], "q: the cache's head dim")
    a.same = (q.shape[1], *k_cache.shape[2:], k_cache.shape[1], dtype)
    a.least = (b, q.shape[0], block_table.shape[1], k_cache.shape[0])
    a.positions = score.shape[2]
    return a


def fp8kv_attn_cache_score(plan: CacheScorePlan, args: CacheScoreArgs, stream: int = 0) -> None:
    _fits(plan, args)
    if args.same is not None:
        _check(args.positions >= plan.max_kv_len, "score: fewer positions than the plan's max_kv_len")
    rc = lib.fp8kv_attn_cache_score(ctypes.byref(plan), ctypes.byref(args), stream)
    if rc != OK:
        raise Fp8kvError(rc, "fp8kv_attn_cache_score")


@dataclass
class CacheScoreCall:
    """Planned gathered weights over fixed device buffers (graph friendly)."""
    plan: CacheScorePlan
    args: CacheScoreArgs

    def run(self, stream: int) -> None:
        fp8kv_attn_cache_score(self.plan, self.args, stream)


def make_cache_select_args(*, score, kv_len, budget: int, keep, n_keep, sinks: int = 0, recent: int = 0,
                           status=None) -> CacheSelectArgs:
    """Fill a CacheSelectArgs struct from torch CUDA tensors.

    score: float32 [B][Hkv][positions]; kv_len, n_keep: int32 [B]; keep: int32
    [B][Hkv][>= min(budget, positions)] for a list per KV head, [B][1][...] for
    one list by the heads' sum; status: optional int32 tensor of one element."""
    _one_device(score, kv_len, keep, n_keep, status)
    a = CacheSelectArgs()
    a.score_stride_req, a.score_stride_head = _weights(score, "score")
    a.keep_stride_req, a.keep_stride_list = _lists(keep, "keep")
    a.batch, a.num_kv_heads, a.max_len = score.shape
    _check(keep.shape[0] == a.batch and keep.shape[1] in (1, a.num_kv_heads) and
           keep.shape[2] >= min(budget, a.max_len), "keep: [B][1 or Hkv][at least min(budget, positions)]")
    _int32(kv_len, a.batch, "kv_len")
    _int32(n_keep, a.batch, "n_keep")
    _status(status)
    a.lists, a.budget, a.sinks, a.recent = keep.shape[1], budget, sinks, recent
    a.score, a.kv_len, a.keep, a.n_keep, a.status = (_ptr(t) for t in (score, kv_len, keep, n_keep, status))
    return a


def fp8kv_attn_cache_select(args: CacheSelectArgs, stream: int = 0) -> None:
    rc = lib.fp8kv_attn_cache_select(ctypes.byref(args), stream)
    if rc != OK:
        raise Fp8kvError(rc, "fp8kv_attn_cache_select")


def make_cache_move_args(*, k_cache, v_cache, block_table, src, count, first=None, dst_table=None, score=None,
                         score_out=None, status=None, kv_format: int = KV_E4M3) -> CacheMoveArgs:
    """Fill a CacheMoveArgs struct from torch CUDA tensors.

    k_cache / v_cache: uint8 [blocks][page][Hkv][D] views (int16 or bfloat16 for
    bf16 caches); block_table, dst_table: int32 [B][columns] (dst_table None: in
    place); src: int32 [B][1 or Hkv][entries], as fp8kv_attn_cache_select writes
    them; count, first: int32 [B] (first None: 0); score / score_out: optional
    float32 [B][Hkv][positions], not overlapping; status: optional int32 tensor of
    one element."""
    _one_device(k_cache, v_cache, block_table, src, count, first, dst_table, score, score_out, status)
    a = CacheMoveArgs()
    size = 2 if kv_format == KV_BF16 else 1
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _check(t.dim() == 4 and t.element_size() == size and t.stride(3) == 1,
               f"{name}: elements of {size} bytes, [blocks][page][Hkv][D] with d contiguous")
    _check(k_cache.shape == v_cache.shape, "v_cache: the same shape as k_cache")
    a.num_kv_blocks, a.page_size, a.num_kv_heads, a.head_dim = k_cache.shape
    a.kv_format = kv_format
    a.block_table, a.block_table_stride = _table(block_table, "block_table")
    a.batch, a.max_blocks = block_table.shape
    if dst_table is not None:
        a.dst_table, a.dst_table_stride = _table(dst_table, "dst_table")
        _check(dst_table.shape[0] == a.batch, "dst_table: a row for each request")
        a.dst_max_blocks = dst_table.shape[1]
    a.src_stride_req, a.src_stride_list = _lists(src, "src")
    _check(src.shape[0] == a.batch and src.shape[1] in (1, a.num_kv_heads), "src: [B][1 or Hkv][entries]")
    a.lists, a.max_count = src.shape[1:]
    _int32(count, a.batch, "count")
    if first is not None:
        _int32(first, a.batch, "first")
    _status(status)
    _check((score is None) == (score_out is None), "score and score_out: both or none")
    if score is not None:
        a.score_stride_req, a.score_stride_head = _weights(score, "score")
        a.score_out_stride_req, a.score_out_stride_head = _weights(score_out, "score_out")
        _check(score.shape == score_out.shape and score.shape[:2] == (a.batch, a.num_kv_heads),
               "score, score_out: [B][Hkv][positions], the same shape")
        a.max_len = score.shape[2]
    a.k_cache, a.v_cache = _ptr(k_cache), _ptr(v_cache)
    a.kc_stride_block, a.kc_stride_token, a.kc_stride_head = (x * size for x in k_cache.stride()[:3])
    a.vc_stride_block, a.vc_stride_token, a.vc_stride_head = (x * size for x in v_cache.stride()[:3])
    a.src, a.count, a.first, a.score, a.score_out, a.status = (
        _ptr(t) for t in (src, count, first, score, score_out, status))
    return a


def fp8kv_attn_cache_move(args: CacheMoveArgs, stream: int = 0) -> None:
    rc = lib.fp8kv_attn_cache_move(ctypes.byref(args), stream)
    if rc != OK:
        raise Fp8kvError(rc, "fp8kv_attn_cache_move")
