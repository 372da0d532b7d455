"""Thin Python binding of ``libkvmm.so`` (the C ABI declared in ``include/kvmm.h``).

Argument marshalling only: every function checks the tensors it is given
(device, dtype, contiguity, element count), turns them into raw device
pointers and calls the C entry point of the same name on the current (or
given) CUDA stream.  All computation happens in the library's kernels; there
is no fallback, and a missing library raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

from . import build as _build

OK, INVALID_ARG, UNSUPPORTED_SHAPE, WORKSPACE_TOO_SMALL, CUDA_ERROR = range(5)
ERR_NULL_BLOCK, ERR_OUT_OF_RANGE, ERR_TIMEOUT = 1, 2, 4
EARLY_READS = DECODE_EARLY_READS = 1
NULL_BLOCK = -1

EXPORTS = ("kv_minmax_update", "page_score_topk", "sparse_paged_decode_attn", "topk_promotion_diff",
           "kvmm_workspace_size", "kvmm_auto_splits", "kvmm_decode_layer_cluster", "kvmm_decode_layer_units",
           "kvmm_status_string",
           "kvmm_last_cuda_error", "page_score_topk_static_scratch", "page_score_topk_attn", "decode_layer", "topk_history_record",
           "topk_stability_rco", "promote_pages", "block_table_update", "kv_meankey_update",
           "page_score_topk_mean", "kv_centroid_build", "page_score_topk_centroid", "kv_append_rope",
           "kv4_append_rope", "kv4_gather", "sparse_paged_decode_attn_kv4", "kvmm_kv4_page_bytes",
           "kvmm_kv4_workspace_size", "sparse_paged_tree_attn", "draft_verify", "kv_keep_path",
           "kvmm_tree_workspace_size")


class KvmmError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = f"{fn}: {status_string(status)} (status {status})"
        if status == CUDA_ERROR:
            msg += f": {load().kvmm_last_cuda_error().decode()}"
        super().__init__(msg)
        self.status = status


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("L", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("D", ctypes.c_int32), ("T", ctypes.c_int32), ("Pmax", ctypes.c_int32), ("Kmax", ctypes.c_int32),
                ("n_phys", ctypes.c_int64)]

    @property
    def G(self) -> int:
        return self.Hq // self.Hkv

    def __repr__(self) -> str:
        return ("Shape(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")")


class Rows(ctypes.Structure):
    """``kvmm_rows``: bf16 rows [batch][token][head] by their strides (in elements)."""

    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class RopeStruct(ctypes.Structure):
    """``kvmm_rope``."""

    _fields_ = [("table", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("rows", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class Rope:
    """The position rotation of kv_append_rope and kv4_append_rope: ``table`` [rows, 2, dim/2] float32 (cosines, then
    sines, of each position), the first ``dim`` channels turned in pairs (i, i + dim/2), or (2i, 2i + 1) with
    ``interleaved``.  ``positions`` [B, n_new] int32: the tokens' positions when they are not their indices; it may be
    replaced between calls, the table stays."""

    def __init__(self, table: torch.Tensor, dim: int, interleaved: bool = False, positions: torch.Tensor | None = None):
        if table.dim() != 3 or table.shape[1] != 2 or table.shape[2] * 2 != dim:
            raise ValueError(f"table must be [rows, 2, {dim // 2}], got {tuple(table.shape)}")
        self._table = table
        self.c = RopeStruct(_dev(table, "table", torch.float32), None, table.shape[0], dim, int(bool(interleaved)))
        self.ref = ctypes.byref(self.c)
        self.positions = positions

    @property
    def table(self) -> torch.Tensor:
        return self._table

    @property
    def dim(self) -> int:
        return self.c.dim

    @property
    def positions(self) -> torch.Tensor | None:
        return self._positions

    @positions.setter
    def positions(self, positions: torch.Tensor | None) -> None:
        # (the struct holds the address that the kernel reads: checked and set together)
        self.c.positions = _dev(positions, "positions", torch.int32, optional=True)
        self._positions = positions


def make_shape(B, L, Hq, Hkv, D, T, Pmax, Kmax, n_phys) -> Shape:
    return Shape(B, L, Hq, Hkv, D, T, Pmax, Kmax, n_phys)


_lib = None


def library_path() -> str:
    return _build.LIB_PATH


def load(path: str | None = None) -> ctypes.CDLL:
    """Load ``libkvmm.so`` (built by ``paged_kv_cache_minmax_gb300.build``); raises if absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    path = path or library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"kvmm CUDA library not found at {path}: build it first "
                           "(python -m paged_kv_cache_minmax_gb300.build)")
    lib = ctypes.CDLL(path)
    P, I32, F32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    SP = ctypes.POINTER(Shape)
    lib.kv_minmax_update.argtypes = [SP, I32, P, P, I32, P, P, P, P, P, P, P, P]
    U32 = ctypes.c_uint32
    lib.page_score_topk.argtypes = [SP, I32, P, P, P, P, I32, I32, P, P, P, P, SZ, U32, P, P]
    lib.sparse_paged_decode_attn.argtypes = [SP, I32, P, P, P, P, P, P, P, F32, I32, P, P, P, SZ, U32, P, P]
    lib.topk_promotion_diff.argtypes = [SP, I32, P, P, P, P, P, I32, P, P, P, P, P, P, P]
    lib.page_score_topk_static_scratch.argtypes = [SP, I32, P, P, P, P, I32, I32, P, P, P, P, P]
    lib.page_score_topk_attn.argtypes = [SP, I32, P, P, P, P, P, P, P, I32, I32, F32, P, P, P, P, P, P, SZ, P, P]
    lib.decode_layer.argtypes = [SP, I32, P, P, P, I32, P, P, P, P, P, P, P, P, I32, I32, F32, P, P, P, P, P, P, SZ,
                                 ctypes.c_uint32, P, P]
    lib.topk_history_record.argtypes = [SP, I32, P, P, P, I32, I32, P, P, P, P, P]
    lib.topk_stability_rco.argtypes = [SP, P, P, P, I32, I32, I32, I32, F32, P, P, P, P, P]
    lib.promote_pages.argtypes = [SP, I32, P, P, P, P, P, P, P, P, P, P, P, P, P, I32, P, P]
    lib.block_table_update.argtypes = [SP, P, P, I32, P, P, P]
    lib.kv_meankey_update.argtypes = [SP, I32, P, P, P, P, P, P, P]
    lib.page_score_topk_mean.argtypes = [SP, I32, P, P, P, P, I32, I32, P, P, P, P, SZ, P, P]
    lib.kv_centroid_build.argtypes = [SP, I32, P, P, I32, I32, P, P, P, P, P, P]
    lib.page_score_topk_centroid.argtypes = [SP, I32, P, P, P, I32, P, P, P, P, I32, I32, I32, P, P, P, P, P, P]
    # kvmm_rows and kvmm_rope by address: packed bytes or a ctypes structure
    lib.kv_append_rope.argtypes = [SP, I32, P, P, P, I32, P, P, P, P, P, P, P, P, P, P]
    lib.kv4_append_rope.argtypes = [SP, I32, P, P, P, I32, P, P, P, P, P, F32, F32, P, P, P, P]
    lib.kv4_gather.argtypes = [SP, I32, P, F32, F32, P, P, P, I32, P, P, P, P]
    lib.sparse_paged_decode_attn_kv4.argtypes = [SP, I32, P, P, F32, F32, P, P, P, P, F32, P, P, P, SZ, U32, P, P]
    lib.kvmm_kv4_page_bytes.argtypes = [SP]
    lib.kvmm_kv4_page_bytes.restype = SZ
    lib.kvmm_kv4_workspace_size.argtypes = [SP]
    lib.kvmm_kv4_workspace_size.restype = SZ
    I64 = ctypes.c_int64
    lib.sparse_paged_tree_attn.argtypes = [SP, I32, P, I32, P, P, P, P, P, P, P, P, F32, P, P, P, SZ, P, P]
    lib.draft_verify.argtypes = [I32, I32, I32, P, I64, P, I64, P, P, P, P, P, I32, P, P, P, P, P]
    lib.kv_keep_path.argtypes = [SP, I32, P, P, I32, P, P, P, P, P, P, P]
    lib.kvmm_tree_workspace_size.argtypes = [SP, I32]
    lib.kvmm_tree_workspace_size.restype = SZ
    for f in ("kv_append_rope", "kv4_append_rope", "kv4_gather", "sparse_paged_decode_attn_kv4",
              "sparse_paged_tree_attn", "draft_verify", "kv_keep_path"):
        getattr(lib, f).restype = ctypes.c_int
    for f in ("kv_minmax_update", "page_score_topk", "sparse_paged_decode_attn", "topk_promotion_diff",
              "page_score_topk_static_scratch", "page_score_topk_attn", "decode_layer", "topk_history_record",
              "topk_stability_rco", "promote_pages", "block_table_update", "kv_meankey_update",
              "page_score_topk_mean", "kv_centroid_build", "page_score_topk_centroid"):
        getattr(lib, f).restype = ctypes.c_int
    lib.kvmm_workspace_size.argtypes = [SP, I32]
    lib.kvmm_workspace_size.restype = SZ
    lib.kvmm_auto_splits.argtypes = [SP]
    lib.kvmm_auto_splits.restype = I32
    lib.kvmm_decode_layer_cluster.argtypes = [SP]
    lib.kvmm_decode_layer_cluster.restype = I32
    lib.kvmm_decode_layer_units.argtypes = [SP]
    lib.kvmm_decode_layer_units.restype = I32
    lib.kvmm_status_string.argtypes = [ctypes.c_int]
    lib.kvmm_status_string.restype = ctypes.c_char_p
    lib.kvmm_last_cuda_error.argtypes = []
    lib.kvmm_last_cuda_error.restype = ctypes.c_char_p
    if path == library_path():
        _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().kvmm_status_string(status).decode()


def _check(fn: str, status: int) -> None:
    if status != OK:
        raise KvmmError(fn, status)


def _dev(t: torch.Tensor | None, name: str, dtype: torch.dtype, numel: int | None = None, optional=False):
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")
    return t.data_ptr()


def _stream(stream) -> int | None:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


# --------------------------------------------------------------------------- #
def workspace_size(shape: Shape, num_splits: int = 0) -> int:
    return int(load().kvmm_workspace_size(ctypes.byref(shape), num_splits))


def auto_splits(shape: Shape) -> int:
    return int(load().kvmm_auto_splits(ctypes.byref(shape)))


def decode_layer_cluster(shape: Shape) -> int:
    return int(load().kvmm_decode_layer_cluster(ctypes.byref(shape)))


def decode_layer_units(shape: Shape) -> int:
    return int(load().kvmm_decode_layer_units(ctypes.byref(shape)))


def alloc_workspace(shape: Shape, num_splits: int = 0, device="cuda") -> torch.Tensor:
    """A zero-filled workspace (uint8) of ``workspace_size`` bytes, rounded to 16."""
    n = workspace_size(shape, num_splits)
    if n == 0:
        raise KvmmError("kvmm_workspace_size", UNSUPPORTED_SHAPE)
    return torch.zeros((n + 15) // 16 * 16, dtype=torch.uint8, device=device)


def kv_minmax_update(shape: Shape, layer: int, new_k, new_v, n_new: int, tok_begin, tok_end, k_pool, v_pool,
                     block_table, meta, err=None, stream=None) -> None:
    s = shape
    if (new_k is None) != (new_v is None):
        raise ValueError("new_k and new_v are given together or not at all")
    rows = s.B * s.Hkv * n_new * s.D
    args = (ctypes.byref(s), layer,
            _dev(new_k, "new_k", torch.bfloat16, rows, optional=True),
            _dev(new_v, "new_v", torch.bfloat16, rows, optional=True), n_new,
            _dev(tok_begin, "tok_begin", torch.int32, s.B), _dev(tok_end, "tok_end", torch.int32, s.B),
            _dev(k_pool, "k_pool", torch.bfloat16, s.n_phys * s.T * s.D),
            _dev(v_pool, "v_pool", torch.bfloat16, s.n_phys * s.T * s.D),
            _dev(block_table, "block_table", torch.int32, s.B * s.L * s.Hkv * s.Pmax),
            _dev(meta, "meta", torch.bfloat16, s.B * s.L * s.Hkv * s.Pmax * 2 * s.D),
            _dev(err, "err", torch.int32, 1, optional=True), _stream(stream))
    _check("kv_minmax_update", load().kv_minmax_update(*args))


def page_score_topk(shape: Shape, layer: int, q, meta, seq_len, rescore_mask, K: int, sel_idx, sel_cnt,
                    workspace, err=None, scores_out=None, group_reduce: int = 0, stream=None,
                    early_reads: bool = False) -> None:
    """Score and select for one layer.  ``early_reads``: no kernel still running when this launch starts
    writes seq_len, the layer's rescore_mask row or its metadata rows (``KVMM_EARLY_READS``)."""
    s = shape
    units = s.B * s.L * s.Hkv
    args = (ctypes.byref(s), layer, _dev(q, "q", torch.bfloat16, s.B * s.Hq * s.D),
            _dev(meta, "meta", torch.bfloat16, units * s.Pmax * 2 * s.D),
            _dev(seq_len, "seq_len", torch.int32, s.B),
            _dev(rescore_mask, "rescore_mask", torch.uint8, s.L * s.Hkv, optional=True), K, group_reduce,
            _dev(sel_idx, "sel_idx", torch.int32, units * s.Kmax), _dev(sel_cnt, "sel_cnt", torch.int32, units),
            _dev(scores_out, "scores_out", torch.float32, s.B * s.Hkv * s.Pmax, optional=True),
            _dev(workspace, "workspace", torch.uint8), workspace.numel(), EARLY_READS if early_reads else 0,
            _dev(err, "err", torch.int32, 1, optional=True), _stream(stream))
    _check("page_score_topk", load().page_score_topk(*args))


def page_score_topk_static_scratch(shape: Shape, layer: int, q, meta, seq_len, rescore_mask, K: int, sel_idx,
                                   sel_cnt, err=None, scores_out=None, group_reduce: int = 0, stream=None) -> None:
    """page_score_topk with the library's fixed device scratch instead of a caller workspace.

    For callers that cannot allocate device memory at call time; the scratch
    is shared by every call on a device, so calls must not overlap on the GPU.
    """
    s = shape
    units = s.B * s.L * s.Hkv
    args = (ctypes.byref(s), layer, _dev(q, "q", torch.bfloat16, s.B * s.Hq * s.D),
            _dev(meta, "meta", torch.bfloat16, units * s.Pmax * 2 * s.D),
            _dev(seq_len, "seq_len", torch.int32, s.B),
            _dev(rescore_mask, "rescore_mask", torch.uint8, s.L * s.Hkv, optional=True), K, group_reduce,
            _dev(sel_idx, "sel_idx", torch.int32, units * s.Kmax), _dev(sel_cnt, "sel_cnt", torch.int32, units),
            _dev(scores_out, "scores_out", torch.float32, s.B * s.Hkv * s.Pmax, optional=True),
            _dev(err, "err", torch.int32, 1, optional=True), _stream(stream))
    _check("page_score_topk_static_scratch", load().page_score_topk_static_scratch(*args))


def sparse_paged_decode_attn(shape: Shape, layer: int, q, k_pool, v_pool, block_table, seq_len, sel_idx, sel_cnt,
                             out, workspace, lse=None, err=None, sm_scale: float = 0.0, num_splits: int = 0,
                             stream=None, early_reads: bool = False) -> None:
    """Attention over the kept selections of one layer.  ``early_reads`` (automatic split count only): no
    kernel still running when this launch starts writes seq_len or the layer's block-table rows."""
    s = shape
    units = s.B * s.L * s.Hkv
    args = (ctypes.byref(s), layer, _dev(q, "q", torch.bfloat16, s.B * s.Hq * s.D),
            _dev(k_pool, "k_pool", torch.bfloat16, s.n_phys * s.T * s.D),
            _dev(v_pool, "v_pool", torch.bfloat16, s.n_phys * s.T * s.D),
            _dev(block_table, "block_table", torch.int32, units * s.Pmax),
            _dev(seq_len, "seq_len", torch.int32, s.B),
            _dev(sel_idx, "sel_idx", torch.int32, units * s.Kmax), _dev(sel_cnt, "sel_cnt", torch.int32, units),
            float(sm_scale), num_splits, _dev(out, "out", torch.float32, s.B * s.Hq * s.D),
            _dev(lse, "lse", torch.float32, s.B * s.Hq, optional=True),
            _dev(workspace, "workspace", torch.uint8, optional=True),
            0 if workspace is None else workspace.numel(), EARLY_READS if early_reads else 0,
            _dev(err, "err", torch.int32, 1, optional=True), _stream(stream))
    _check("sparse_paged_decode_attn", load().sparse_paged_decode_attn(*args))


def page_score_topk_attn(shape: Shape, layer: int, q, meta, k_pool, v_pool, block_table, seq_len, rescore_mask,
                         K: int, sel_idx, sel_cnt, out, workspace, lse=None, err=None, scores_out=None,
                         group_reduce: int = 0, sm_scale: float = 0.0, stream=None) -> None:
    """page_score_topk then sparse_paged_decode_attn on the new selection, in one launch."""
    s = shape
    units = s.B * s.L * s.Hkv
    args = (ctypes.byref(s), layer, _dev(q, "q", torch.bfloat16, s.B * s.Hq * s.D),
            _dev(meta, "meta", torch.bfloat16, units * s.Pmax * 2 * s.D),
            _dev(k_pool, "k_pool", torch.bfloat16, s.n_phys * s.T * s.D),
            _dev(v_pool, "v_pool", torch.bfloat16, s.n_phys * s.T * s.D),
            _dev(block_table, "block_table", torch.int32, units * s.Pmax),
            _dev(seq_len, "seq_len", torch.int32, s.B),
            _dev(rescore_mask, "rescore_mask", torch.uint8, s.L * s.Hkv, optional=True), K, group_reduce,
            float(sm_scale),
            _dev(sel_idx, "sel_idx", torch.int32, units * s.Kmax), _dev(sel_cnt, "sel_cnt", torch.int32, units),
            _dev(scores_out, "scores_out", torch.float32, s.B * s.Hkv * s.Pmax, optional=True),
            _dev(out, "out", torch.float32, s.B * s.Hq * s.D),
            _dev(lse, "lse", torch.float32, s.B * s.Hq, optional=True),
            _dev(workspace, "workspace", torch.uint8), workspace.numel(),
            _dev(err, "err", torch.int32, 1, optional=True), _stream(stream))
    _check("page_score_topk_attn", load().page_score_topk_attn(*args))


def decode_layer(shape: Shape, layer: int, q, new_k, new_v, n_new: int, tok_begin, tok_end, k_pool, v_pool,
                 block_table, meta, seq_len, rescore_mask, K: int, sel_idx, sel_cnt, out, lse=None, err=None,
                 scores_out=None, group_reduce: int = 0, sm_scale: float = 0.0, workspace=None,
                 stream=None, early_reads: bool = False) -> None:
    """Append (optional), score, select and attend for one layer in one launch.  ``early_reads``: no kernel
    still running when this launch starts (after a kvmm call: that call alone) writes anything this call reads
    of seq_len, tok_begin, tok_end, rescore_mask, block_table and meta (``KVMM_DECODE_EARLY_READS``); two
    calls for the same layer back to back do not meet this."""
    s = shape
    units = s.B * s.L * s.Hkv
    if (new_k is None) != (new_v is None):
        raise ValueError("new_k and new_v are given together or not at all")
    app = new_k is not None
    args = (ctypes.byref(s), layer, _dev(q, "q", torch.bfloat16, s.B * s.Hq * s.D),
            _dev(new_k, "new_k", torch.bfloat16, s.B * s.Hkv * max(n_new, 1) * s.D, optional=True),
            _dev(new_v, "new_v", torch.bfloat16, s.B * s.Hkv * max(n_new, 1) * s.D, optional=True),
            int(n_new) if app else 0,
            _dev(tok_begin, "tok_begin", torch.int32, s.B, optional=not app),
            _dev(tok_end, "tok_end", torch.int32, s.B, optional=not app),
            _dev(k_pool, "k_pool", torch.bfloat16, s.n_phys * s.T * s.D),
            _dev(v_pool, "v_pool", torch.bfloat16, s.n_phys * s.T * s.D),
            _dev(block_table, "block_table", torch.int32, units * s.Pmax),
            _dev(meta, "meta", torch.bfloat16, units * s.Pmax * 2 * s.D),
            _dev(seq_len, "seq_len", torch.int32, s.B),
            _dev(rescore_mask, "rescore_mask", torch.uint8, s.L * s.Hkv, optional=True), K, group_reduce,
            float(sm_scale),
            _dev(sel_idx, "sel_idx", torch.int32, units * s.Kmax), _dev(sel_cnt, "sel_cnt", torch.int32, units),
            _dev(scores_out, "scores_out", torch.float32, s.B * s.Hkv * s.Pmax, optional=True),
            _dev(out, "out", torch.float32, s.B * s.Hq * s.D),
            _dev(lse, "lse", torch.float32, s.B * s.Hq, optional=True),
            _dev(workspace, "workspace", torch.uint8, optional=True), 0 if workspace is None else workspace.numel(),
            DECODE_EARLY_READS if early_reads else 0,
            _dev(err, "err", torch.int32, 1, optional=True), _stream(stream))
    _check("decode_layer", load().decode_layer(*args))


def topk_promotion_diff(shape: Shape, layer: int, rescore_mask, prev_idx, prev_cnt, cur_idx, cur_cnt, promoted,
                        promoted_cnt, evicted=None, evicted_cnt=None, total_promoted=None, commit: bool = True,
                        err=None, stream=None) -> None:
    s = shape
    units = s.B * s.L * s.Hkv
    args = (ctypes.byref(s), layer,
            _dev(rescore_mask, "rescore_mask", torch.uint8, s.L * s.Hkv, optional=True),
            _dev(prev_idx, "prev_idx", torch.int32, units * s.Kmax), _dev(prev_cnt, "prev_cnt", torch.int32, units),
            _dev(cur_idx, "cur_idx", torch.int32, units * s.Kmax), _dev(cur_cnt, "cur_cnt", torch.int32, units),
            int(bool(commit)), _dev(promoted, "promoted", torch.int32, units * s.Kmax),
            _dev(promoted_cnt, "promoted_cnt", torch.int32, units),
            _dev(evicted, "evicted", torch.int32, units * s.Kmax, optional=True),
            _dev(evicted_cnt, "evicted_cnt", torch.int32, units, optional=True),
            _dev(total_promoted, "total_promoted", torch.int32, 1, optional=True),
            _dev(err, "err", torch.int32, 1, optional=True), _stream(stream))
    _check("topk_promotion_diff", load().topk_promotion_diff(*args))


def topk_history_record(shape: Shape, layer: int, sel_idx, sel_cnt, seq_len, slot: int, hist_idx, hist_cnt,
                        hist_pages, err=None, stream=None) -> None:
    """Store ``layer``'s selections in ring slot ``slot`` (hist_idx [W,B,L,Hkv,Kmax], hist_cnt [W,B,L,Hkv],
    hist_pages [W,B], all int32; W is taken from hist_pages)."""
    s = shape
    units = s.B * s.L * s.Hkv
    W = hist_pages.shape[0]
    args = (ctypes.byref(s), layer, _dev(sel_idx, "sel_idx", torch.int32, units * s.Kmax),
            _dev(sel_cnt, "sel_cnt", torch.int32, units), _dev(seq_len, "seq_len", torch.int32, s.B), W, slot,
            _dev(hist_idx, "hist_idx", torch.int32, W * units * s.Kmax),
            _dev(hist_cnt, "hist_cnt", torch.int32, W * units), _dev(hist_pages, "hist_pages", torch.int32, W * s.B),
            _dev(err, "err", torch.int32, 1, optional=True), _stream(stream))
    _check("topk_history_record", load().topk_history_record(*args))


def topk_stability_rco(shape: Shape, hist_idx, hist_cnt, hist_pages, n: int, head: int, lag: int, rco_unit,
                       stability=None, unstable=None, unstable_frac: float = 0.25, err=None, stream=None) -> None:
    """Per-unit mean RCO of selections ``lag`` steps apart over the last ``n`` recorded steps (newest in slot
    ``head``), the per-head stability and the unstable mask; see kvmm.h."""
    s = shape
    units = s.B * s.L * s.Hkv
    W = hist_pages.shape[0]
    args = (ctypes.byref(s), _dev(hist_idx, "hist_idx", torch.int32, W * units * s.Kmax),
            _dev(hist_cnt, "hist_cnt", torch.int32, W * units), _dev(hist_pages, "hist_pages", torch.int32, W * s.B),
            W, n, head, lag, float(unstable_frac), _dev(rco_unit, "rco_unit", torch.float32, units),
            _dev(stability, "stability", torch.float32, s.L * s.Hkv, optional=True),
            _dev(unstable, "unstable", torch.uint8, s.L * s.Hkv, optional=True),
            _dev(err, "err", torch.int32, 1, optional=True), _stream(stream))
    _check("topk_stability_rco", load().topk_stability_rco(*args))


def _host(t: torch.Tensor, name: str, numel: int):
    """A host-side bf16 store (pinned, or pageable where the device reads pageable memory)."""
    if t.is_cuda:
        raise ValueError(f"{name} must be a host tensor")
    if t.dtype != torch.bfloat16 or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous bfloat16")
    if t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")
    return t.data_ptr()


def promote_pages(shape: Shape, layer: int, rescore_mask, promoted, promoted_cnt, evicted, evicted_cnt, host_k,
                  host_v, k_pool, v_pool, block_table, moved=None, freed=None, freed_cnt=None, max_ctas: int = 0,
                  err=None, stream=None) -> None:
    """Promoted pages from the host store (host_k [B,L,Hkv,Pmax,T,D], host_v [B,L,Hkv,Pmax,D,T], bf16) into the
    blocks of evicted pages, and the table rewrite; see kvmm.h."""
    s = shape
    units = s.B * s.L * s.Hkv
    page = s.T * s.D
    args = (ctypes.byref(s), layer, _dev(rescore_mask, "rescore_mask", torch.uint8, s.L * s.Hkv, optional=True),
            _dev(promoted, "promoted", torch.int32, units * s.Kmax),
            _dev(promoted_cnt, "promoted_cnt", torch.int32, units),
            _dev(evicted, "evicted", torch.int32, units * s.Kmax), _dev(evicted_cnt, "evicted_cnt", torch.int32, units),
            _host(host_k, "host_k", units * s.Pmax * page), _host(host_v, "host_v", units * s.Pmax * page),
            _dev(k_pool, "k_pool", torch.bfloat16, s.n_phys * page), _dev(v_pool, "v_pool", torch.bfloat16, s.n_phys * page),
            _dev(block_table, "block_table", torch.int32, units * s.Pmax),
            _dev(moved, "moved", torch.int32, units, optional=True),
            _dev(freed, "freed", torch.int32, units * s.Kmax, optional=True),
            _dev(freed_cnt, "freed_cnt", torch.int32, units, optional=True), int(max_ctas),
            _dev(err, "err", torch.int32, 1, optional=True), _stream(stream))
    _check("promote_pages", load().promote_pages(*args))


def block_table_update(shape: Shape, idx, val, block_table, err=None, stream=None) -> None:
    """block_table.view(-1)[idx[i]] = val[i]; idx (int64) and val (int32) on the device or in pinned host memory."""
    s = shape
    n = int(idx.numel())
    if int(val.numel()) != n:
        raise ValueError("idx and val differ in length")
    for t, name, dt in ((idx, "idx", torch.int64), (val, "val", torch.int32)):
        if t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous {dt}")
    args = (ctypes.byref(s), idx.data_ptr() if n else None, val.data_ptr() if n else None, n,
            _dev(block_table, "block_table", torch.int32, s.B * s.L * s.Hkv * s.Pmax),
            _dev(err, "err", torch.int32, 1, optional=True), _stream(stream))
    _check("block_table_update", load().block_table_update(*args))


def kv_meankey_update(shape: Shape, layer: int, tok_begin, tok_end, k_pool, block_table, mean, err=None,
                      stream=None) -> None:
    """Mean key of every page meeting [tok_begin, tok_end) (tok_begin None = 0) into mean [B,L,Hkv,Pmax,D]."""
    s = shape
    units = s.B * s.L * s.Hkv
    args = (ctypes.byref(s), layer, _dev(tok_begin, "tok_begin", torch.int32, s.B, optional=True),
            _dev(tok_end, "tok_end", torch.int32, s.B), _dev(k_pool, "k_pool", torch.bfloat16, s.n_phys * s.T * s.D),
            _dev(block_table, "block_table", torch.int32, units * s.Pmax),
            _dev(mean, "mean", torch.bfloat16, units * s.Pmax * s.D), _dev(err, "err", torch.int32, 1, optional=True),
            _stream(stream))
    _check("kv_meankey_update", load().kv_meankey_update(*args))


def page_score_topk_mean(shape: Shape, layer: int, q, mean, seq_len, rescore_mask, K: int, sel_idx, sel_cnt,
                         workspace, err=None, scores_out=None, group_reduce: int = 0, stream=None) -> None:
    """page_score_topk with the mean key (mean [B,L,Hkv,Pmax,D]) as the page's row."""
    s = shape
    units = s.B * s.L * s.Hkv
    args = (ctypes.byref(s), layer, _dev(q, "q", torch.bfloat16, s.B * s.Hq * s.D),
            _dev(mean, "mean", torch.bfloat16, units * s.Pmax * s.D),
            _dev(seq_len, "seq_len", torch.int32, s.B),
            _dev(rescore_mask, "rescore_mask", torch.uint8, s.L * s.Hkv, optional=True), K, group_reduce,
            _dev(sel_idx, "sel_idx", torch.int32, units * s.Kmax), _dev(sel_cnt, "sel_cnt", torch.int32, units),
            _dev(scores_out, "scores_out", torch.float32, s.B * s.Hkv * s.Pmax, optional=True),
            _dev(workspace, "workspace", torch.uint8), workspace.numel(),
            _dev(err, "err", torch.int32, 1, optional=True), _stream(stream))
    _check("page_score_topk_mean", load().page_score_topk_mean(*args))


def centroid_rows(shape: Shape, R: int) -> int:
    """Cmax = ceil(Pmax / R): the centroid rows a unit holds at most."""
    return (shape.Pmax + R - 1) // R


def kv_centroid_build(shape: Shape, layer: int, mean, seq_len, R: int, n_iter: int, cent, assign, member_off, members,
                      err=None, stream=None) -> None:
    """KVDrive's centroid level over the layer's pages' mean keys: spatial blocks of R pages, then n_iter Lloyd
    iterations.  cent [B,L,Hkv,Cmax,D] bf16, assign [B,L,Hkv,Pmax], member_off [B,L,Hkv,Cmax+1],
    members [B,L,Hkv,Pmax] int32 (Cmax = ceil(Pmax / R))."""
    s = shape
    units = s.B * s.L * s.Hkv
    cmax = centroid_rows(s, R)
    args = (ctypes.byref(s), layer, _dev(mean, "mean", torch.bfloat16, units * s.Pmax * s.D),
            _dev(seq_len, "seq_len", torch.int32, s.B), int(R), int(n_iter),
            _dev(cent, "cent", torch.bfloat16, units * cmax * s.D), _dev(assign, "assign", torch.int32, units * s.Pmax),
            _dev(member_off, "member_off", torch.int32, units * (cmax + 1)),
            _dev(members, "members", torch.int32, units * s.Pmax), _dev(err, "err", torch.int32, 1, optional=True),
            _stream(stream))
    _check("kv_centroid_build", load().kv_centroid_build(*args))


def page_score_topk_centroid(shape: Shape, layer: int, q, mean, seq_len, R: int, cent, member_off, members,
                             rescore_mask, M: int, K: int, sel_idx, sel_cnt, err=None, centroid_scores_out=None,
                             scores_out=None, group_reduce: int = 0, stream=None) -> None:
    """The two-level selection: score the centroids, expand the M best, keep the K best of their pages."""
    s = shape
    units = s.B * s.L * s.Hkv
    cmax = centroid_rows(s, R)
    args = (ctypes.byref(s), layer, _dev(q, "q", torch.bfloat16, s.B * s.Hq * s.D),
            _dev(mean, "mean", torch.bfloat16, units * s.Pmax * s.D), _dev(seq_len, "seq_len", torch.int32, s.B),
            int(R), _dev(cent, "cent", torch.bfloat16, units * cmax * s.D),
            _dev(member_off, "member_off", torch.int32, units * (cmax + 1)),
            _dev(members, "members", torch.int32, units * s.Pmax),
            _dev(rescore_mask, "rescore_mask", torch.uint8, s.L * s.Hkv, optional=True), int(M), int(K),
            int(group_reduce), _dev(sel_idx, "sel_idx", torch.int32, units * s.Kmax),
            _dev(sel_cnt, "sel_cnt", torch.int32, units),
            _dev(centroid_scores_out, "centroid_scores_out", torch.float32, s.B * s.Hkv * cmax, optional=True),
            _dev(scores_out, "scores_out", torch.float32, s.B * s.Hkv * s.Pmax, optional=True),
            _dev(err, "err", torch.int32, 1, optional=True), _stream(stream))
    _check("page_score_topk_centroid", load().page_score_topk_centroid(*args))


# --------------------------------------------------------------------------- #
def kv4_page_bytes(shape: Shape) -> int:
    """Bytes of one page of the 4-bit cache (keys and values, codes and scales)."""
    return int(load().kvmm_kv4_page_bytes(ctypes.byref(shape)))


def kv4_workspace_size(shape: Shape) -> int:
    return int(load().kvmm_kv4_workspace_size(ctypes.byref(shape)))


def alloc_kv4_pool(shape: Shape, device="cuda") -> torch.Tensor:
    """A zero-filled pool [n_phys, page bytes] (uint8) of the 4-bit cache."""
    n = kv4_page_bytes(shape)
    if n == 0:
        raise KvmmError("kvmm_kv4_page_bytes", UNSUPPORTED_SHAPE)
    return torch.zeros(shape.n_phys, n, dtype=torch.uint8, device=device)


def alloc_kv4_workspace(shape: Shape, device="cuda") -> torch.Tensor:
    """A workspace (uint8, zero-filled as it has to be) for sparse_paged_decode_attn_kv4."""
    n = kv4_workspace_size(shape)
    if n == 0:
        raise KvmmError("kvmm_kv4_workspace_size", UNSUPPORTED_SHAPE)
    return torch.zeros((n + 15) // 16 * 16, dtype=torch.uint8, device=device)


_fields = struct.Struct("8iq").unpack_from  # a Shape's fields at once: single ones cost a small call its time
_pack_rows = struct.Struct("Pqqq").pack     # a kvmm_rows


def _here(stream) -> tuple[int, int]:
    """The current device and the stream of a call: every tensor of the call has to be on that device."""
    here = torch.cuda.current_device()
    return here, torch._C._cuda_getCurrentRawStream(here) if stream is None else stream.cuda_stream


def _arg(t: torch.Tensor, name: str, dtype: torch.dtype, numel: int, here: int) -> int:
    """_dev, and the tensor is on the call's device."""
    if t is None or t.get_device() != here or t.dtype is not dtype or not t.is_contiguous() or t.numel() < numel:
        _dev(t, name, dtype, numel)
        raise ValueError(f"{name} is on {t.device}, the call on cuda:{here}")
    return t.data_ptr()


def _opt(t: torch.Tensor | None, name: str, dtype: torch.dtype, numel: int, here: int) -> int | None:
    return None if t is None else _arg(t, name, dtype, numel, here)


def _rows(t: torch.Tensor, name: str, B: int, n: int, H: int, D: int, here: int) -> bytes:
    """A [B, n, H, D] bf16 view as a kvmm_rows."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != here:
        raise ValueError(f"{name} is on {t.device}, the call on cuda:{here}")
    if t.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.shape != (B, n, H, D):
        raise ValueError(f"{name} must be {(B, n, H, D)}, got {tuple(t.shape)}")
    sb, st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name}: the channels of a row must be consecutive")
    # an axis of one entry has no step: its stride may be anything
    return _pack_rows(t.data_ptr(), sb if B > 1 else 0, st if n > 1 else 0, sh if H > 1 else 0)


def _dense(t: torch.Tensor, name: str, shape: tuple[int, ...]) -> None:
    """The axes of a dense t step as those of [shape] do: one with longer rows, or rows in another order, holds them
    elsewhere, however many elements it has."""
    if t.shape == shape:
        return
    steps, step = {1}, 1
    for n in reversed(shape[1:]):
        step *= n
        steps.add(step)
    if any(n > 1 and st not in steps for n, st in zip(t.shape, t.stride())):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _append_rows(f, q, new_k, new_v, tok_begin, tok_end, rope, q_out, here):
    """The arguments kv_append_rope and kv4_append_rope share, from q to q_out."""
    B, _, Hq, Hkv, D = f[:5]
    n = new_k.shape[1] if new_k.dim() == 4 else -1
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out are given together or not at all")
    if rope is not None:
        if rope.table.get_device() != here:
            raise ValueError(f"the rope's table is on {rope.table.device}, the call on cuda:{here}")
        if rope.positions is not None and (rope.positions.numel() < B * n or rope.positions.get_device() != here):
            raise ValueError(f"positions needs {B * n} elements on cuda:{here}")
        if rope.positions is not None:
            _dense(rope.positions, "positions", (B, n))
    if q_out is not None and (n != 1 or q_out.shape != (B, Hq, D)):
        _dense(q_out, "q_out", (B, n, Hq, D))
    return (None if q is None else _rows(q, "q", B, n, Hq, D, here), _rows(new_k, "new_k", B, n, Hkv, D, here),
            _rows(new_v, "new_v", B, n, Hkv, D, here), n, _arg(tok_begin, "tok_begin", torch.int32, B, here),
            _arg(tok_end, "tok_end", torch.int32, B, here), None if rope is None else rope.ref,
            _opt(q_out, "q_out", torch.bfloat16, B * n * Hq * D, here))


def kv_append_rope(shape: Shape, layer: int, q, new_k, new_v, tok_begin, tok_end, k_pool, v_pool, block_table, meta,
                   rope: Rope | None = None, q_out=None, err=None, stream=None) -> None:
    """Rotate the new tokens' queries and keys, append keys and values, refresh the MinMax of their pages.

    new_k, new_v [B, n_new, Hkv, D] and q [B, n_new, Hq, D] (or None) are bf16 views of any strides whose channels are
    consecutive; q_out [B, n_new, Hq, D] takes the rotated queries; meta may be None."""
    f = _fields(shape)
    B, L, _, Hkv, D, T, Pmax, _, n_phys = f
    here, st = _here(stream)
    pages = B * L * Hkv * Pmax
    status = load().kv_append_rope(
        ctypes.byref(shape), layer, *_append_rows(f, q, new_k, new_v, tok_begin, tok_end, rope, q_out, here),
        _arg(k_pool, "k_pool", torch.bfloat16, n_phys * T * D, here),
        _arg(v_pool, "v_pool", torch.bfloat16, n_phys * T * D, here),
        _arg(block_table, "block_table", torch.int32, pages, here),
        _opt(meta, "meta", torch.bfloat16, pages * 2 * D, here), _opt(err, "err", torch.int32, 1, here), st)
    _check("kv_append_rope", status)


def kv4_append_rope(shape: Shape, layer: int, q, new_k, new_v, tok_begin, tok_end, kv4_pool, block_table, meta,
                    rope: Rope | None = None, q_out=None, k_scale: float = 1.0, v_scale: float = 1.0, err=None,
                    stream=None) -> None:
    """kv_append_rope into the 4-bit cache (kv4_pool [n_phys, kv4_page_bytes] uint8); meta are the bounds of the keys
    as held, over k_scale."""
    f = _fields(shape)
    B, L, _, Hkv, D, T, Pmax, _, n_phys = f
    here, st = _here(stream)
    pages = B * L * Hkv * Pmax
    status = load().kv4_append_rope(
        ctypes.byref(shape), layer, *_append_rows(f, q, new_k, new_v, tok_begin, tok_end, rope, q_out, here),
        _arg(kv4_pool, "kv4_pool", torch.uint8, n_phys * T * (D + D // 8), here), k_scale, v_scale,
        _arg(block_table, "block_table", torch.int32, pages, here),
        _opt(meta, "meta", torch.bfloat16, pages * 2 * D, here), _opt(err, "err", torch.int32, 1, here), st)
    _check("kv4_append_rope", status)


def kv4_gather(shape: Shape, layer: int, kv4_pool, block_table, tok_begin, tok_end, k_out, v_out, k_scale: float = 1.0,
               v_scale: float = 1.0, err=None, stream=None) -> None:
    """Tokens [tok_begin, tok_end) of every KV head (tok_begin None = 0) as bf16 rows of k_out and v_out
    [B, n_rows, Hkv, D] (either may be None); rows behind a sequence's last are left as they were."""
    B, L, _, Hkv, D, T, Pmax, _, n_phys = _fields(shape)
    some = k_out if k_out is not None else v_out
    if some is None:
        raise ValueError("k_out or v_out is required")
    n = some.shape[1] if some.dim() == 4 else -1
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        if t is not None and t.shape != (B, n, Hkv, D):
            raise ValueError(f"{name} must be [{B}, n_rows, {Hkv}, {D}], got {tuple(t.shape)}")
    here, st = _here(stream)
    status = load().kv4_gather(
        ctypes.byref(shape), layer, _arg(kv4_pool, "kv4_pool", torch.uint8, n_phys * T * (D + D // 8), here), k_scale,
        v_scale, _arg(block_table, "block_table", torch.int32, B * L * Hkv * Pmax, here),
        _opt(tok_begin, "tok_begin", torch.int32, B, here), _arg(tok_end, "tok_end", torch.int32, B, here), n,
        _opt(k_out, "k_out", torch.bfloat16, 0, here), _opt(v_out, "v_out", torch.bfloat16, 0, here),
        _opt(err, "err", torch.int32, 1, here), st)
    _check("kv4_gather", status)


def sparse_paged_decode_attn_kv4(shape: Shape, layer: int, q, kv4_pool, block_table, seq_len, sel_idx, sel_cnt, out,
                                 workspace, lse=None, err=None, k_scale: float = 1.0, v_scale: float = 1.0,
                                 sm_scale: float = 0.0, stream=None, early_reads: bool = False) -> None:
    """Attention over the selected pages of the 4-bit cache, or, with sel_idx and sel_cnt None, over every page.
    workspace: alloc_kv4_workspace; calls that may run at once need one each.  ``early_reads``: no kernel still running
    when this launch starts writes seq_len or the layer's block-table rows (used over every page alone)."""
    B, L, Hq, Hkv, D, T, Pmax, Kmax, n_phys = _fields(shape)
    if (sel_idx is None) != (sel_cnt is None):
        raise ValueError("sel_idx and sel_cnt are given together or not at all")
    here, st = _here(stream)
    units = B * L * Hkv
    status = load().sparse_paged_decode_attn_kv4(
        ctypes.byref(shape), layer, _arg(q, "q", torch.bfloat16, B * Hq * D, here),
        _arg(kv4_pool, "kv4_pool", torch.uint8, n_phys * T * (D + D // 8), here), k_scale, v_scale,
        _arg(block_table, "block_table", torch.int32, units * Pmax, here),
        _arg(seq_len, "seq_len", torch.int32, B, here), _opt(sel_idx, "sel_idx", torch.int32, units * Kmax, here),
        _opt(sel_cnt, "sel_cnt", torch.int32, units, here), sm_scale, _arg(out, "out", torch.float32, B * Hq * D, here),
        _opt(lse, "lse", torch.float32, B * Hq, here), _arg(workspace, "workspace", torch.uint8, 0, here),
        workspace.numel(), EARLY_READS if early_reads else 0, _opt(err, "err", torch.int32, 1, here), st)
    _check("sparse_paged_decode_attn_kv4", status)


# --------------------------------------------------------------------------- #
def tree_workspace_size(shape: Shape, n_max: int) -> int:
    return int(load().kvmm_tree_workspace_size(ctypes.byref(shape), n_max))


def alloc_tree_workspace(shape: Shape, n_max: int, device="cuda") -> torch.Tensor:
    """A workspace (uint8) for sparse_paged_tree_attn with up to ``n_max`` nodes a sequence."""
    n = tree_workspace_size(shape, n_max)
    if n == 0:
        raise KvmmError("kvmm_tree_workspace_size", UNSUPPORTED_SHAPE)
    return torch.empty((n + 15) // 16 * 16, dtype=torch.uint8, device=device)


def tree_masks(parent: torch.Tensor) -> torch.Tensor:
    """The tree_mask [B, n] (int64, bit j of node i: i sees j) in which every node sees itself and its ancestors, from
    parent [B, n] (node 0 is the root; parent[:, i] < i; a node with a parent that is no earlier one sees itself alone, or
    with a parent below 0 the root too).  A few launches for each node: for trees that are kept."""
    if parent.dim() != 2 or not 1 <= parent.shape[1] <= 64:
        raise ValueError(f"parent must be [B, n] with 1 <= n <= 64, got {tuple(parent.shape)}")
    n = parent.shape[1]
    up = parent.long().clamp(0, n - 1)  # (a node that is not reached yet has no bits)
    bits = torch.zeros(parent.shape, dtype=torch.int64, device=parent.device)
    for i in range(n):
        own = 1 << i if i < 63 else -(1 << 63)
        bits[:, i] = bits.gather(1, up[:, i:i + 1]).squeeze(1) | own if i else own
    return bits


def _int_rows(t: torch.Tensor, name: str, B: int, n: int, here: int) -> int:
    """A dense [B, n] int32 tensor."""
    if t is None or t.shape != (B, n):
        raise ValueError(f"{name} must be [{B}, {n}], got {None if t is None else list(t.shape)}")
    return _arg(t, name, torch.int32, B * n, here)


def sparse_paged_tree_attn(shape: Shape, layer: int, q, k_pool, v_pool, block_table, seq_len, out, workspace,
                           n_nodes=None, tree_mask=None, sel_idx=None, sel_cnt=None, lse=None, err=None,
                           sm_scale: float = 0.0, stream=None) -> None:
    """Attention of a tree of n nodes a sequence (q, out [B, n, Hq, D] bf16, lse [B, n, Hq]): each node over the settled
    tokens of the selected pages (every page with sel_idx and sel_cnt None) and over the nodes that tree_mask [B, n]
    int64 shows it (``tree_masks``; None: a chain).  The nodes stand at the tokens seq_len + i.  workspace:
    alloc_tree_workspace; calls that may run at once need one each."""
    B, L, Hq, Hkv, D, T, Pmax, Kmax, n_phys = _fields(shape)
    if (sel_idx is None) != (sel_cnt is None):
        raise ValueError("sel_idx and sel_cnt are given together or not at all")
    n = q.shape[1] if q.dim() == 4 else -1
    for t, name in ((q, "q"), (out, "out")):
        if t.shape != (B, n, Hq, D):
            raise ValueError(f"{name} must be [{B}, n, {Hq}, {D}], got {list(t.shape)}")
    if lse is not None and lse.shape != (B, n, Hq):
        raise ValueError(f"lse must be [{B}, {n}, {Hq}], got {list(lse.shape)}")
    if tree_mask is not None and tree_mask.shape != (B, n):
        raise ValueError(f"tree_mask must be [{B}, {n}], got {list(tree_mask.shape)}")
    here, st = _here(stream)
    units = B * L * Hkv
    status = load().sparse_paged_tree_attn(
        ctypes.byref(shape), layer, _arg(q, "q", torch.bfloat16, 0, here), n,
        _opt(n_nodes, "n_nodes", torch.int32, B, here), _opt(tree_mask, "tree_mask", torch.int64, 0, here),
        _arg(k_pool, "k_pool", torch.bfloat16, n_phys * T * D, here),
        _arg(v_pool, "v_pool", torch.bfloat16, n_phys * T * D, here),
        _arg(block_table, "block_table", torch.int32, units * Pmax, here),
        _arg(seq_len, "seq_len", torch.int32, B, here), _opt(sel_idx, "sel_idx", torch.int32, units * Kmax, here),
        _opt(sel_cnt, "sel_cnt", torch.int32, units, here), sm_scale, _arg(out, "out", torch.bfloat16, 0, here),
        _opt(lse, "lse", torch.float32, 0, here), _arg(workspace, "workspace", torch.uint8, 0, here),
        workspace.numel(), _opt(err, "err", torch.int32, 1, here), st)
    _check("sparse_paged_tree_attn", status)


def _prob_rows(t: torch.Tensor, name: str, B: int, n: int, V: int, here: int) -> tuple[int, int]:
    """The address of [B, n, V] float rows a constant step apart, and that step."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != here:
        raise ValueError(f"{name} is on {t.device}, the call on cuda:{here}")
    if t.dtype is not torch.float32:
        raise ValueError(f"{name} must be {torch.float32}, got {t.dtype}")
    if t.shape != (B, n, V):
        raise ValueError(f"{name} must be {(B, n, V)}, got {tuple(t.shape)}")
    sb, sn, sv = t.stride()
    step = sn if n > 1 else sb if B > 1 else V  # an axis of one entry has no step: its stride may be anything
    if (sv != 1 and V > 1) or (n > 1 and B > 1 and sb != n * sn) or step < V:
        raise ValueError(f"{name}: the probabilities of a row must be consecutive and the rows evenly spaced")
    return t.data_ptr(), step


def draft_verify(target_probs, tokens, parent, u_accept, u_next, path, path_len, out_tokens, draft_probs=None,
                 n_nodes=None, distinct: bool = False, err=None, stream=None) -> None:
    """Walk each sequence's tree along accepted nodes and draw the token behind them (see kvmm.h for the rule).

    target_probs, draft_probs [B, n, V] float32 (rows may be padded; draft_probs None: candidates proposed with
    certainty); tokens, parent [B, n] int32; u_accept [B, n], u_next [B] float32 in [0, 1); path, out_tokens [B, n] and
    path_len [B] int32 are written.  ``distinct``: a node's children were drawn without replacement."""
    if target_probs.dim() != 3:
        raise ValueError(f"target_probs must be [B, n, V], got {list(target_probs.shape)}")
    B, n, V = target_probs.shape
    here, st = _here(stream)
    target, tstep = _prob_rows(target_probs, "target_probs", B, n, V, here)
    draft, dstep = (None, 0) if draft_probs is None else _prob_rows(draft_probs, "draft_probs", B, n, V, here)
    if u_accept.shape != (B, n):
        raise ValueError(f"u_accept must be [{B}, {n}], got {list(u_accept.shape)}")
    status = load().draft_verify(
        B, n, V, target, tstep, draft, dstep, _int_rows(tokens, "tokens", B, n, here),
        _int_rows(parent, "parent", B, n, here), _opt(n_nodes, "n_nodes", torch.int32, B, here),
        _arg(u_accept, "u_accept", torch.float32, 0, here), _arg(u_next, "u_next", torch.float32, B, here),
        int(bool(distinct)), _int_rows(path, "path", B, n, here), _arg(path_len, "path_len", torch.int32, B, here),
        _int_rows(out_tokens, "out_tokens", B, n, here), _opt(err, "err", torch.int32, 1, here), st)
    _check("draft_verify", status)


def kv_keep_path(shape: Shape, layer: int, path, path_len, seq_len, k_pool, v_pool, block_table, meta=None, err=None,
                 stream=None) -> None:
    """Move the rows of the accepted nodes path [B, n] (path_len [B] of them) to the tokens seq_len + 0, 1, .. and take
    the MinMax of the pages there again, in ``layer`` or, with -1, in every layer.  seq_len stays as it was."""
    B, L, _, Hkv, D, T, Pmax, _, n_phys = _fields(shape)
    if path.dim() != 2:
        raise ValueError(f"path must be [{B}, n], got {list(path.shape)}")
    n = path.shape[1]
    here, st = _here(stream)
    pages = B * L * Hkv * Pmax
    status = load().kv_keep_path(
        ctypes.byref(shape), layer, _int_rows(path, "path", B, n, here),
        _arg(path_len, "path_len", torch.int32, B, here), n, _arg(seq_len, "seq_len", torch.int32, B, here),
        _arg(k_pool, "k_pool", torch.bfloat16, n_phys * T * D, here),
        _arg(v_pool, "v_pool", torch.bfloat16, n_phys * T * D, here),
        _arg(block_table, "block_table", torch.int32, pages, here),
        _opt(meta, "meta", torch.bfloat16, pages * 2 * D, here), _opt(err, "err", torch.int32, 1, here), st)
    _check("kv_keep_path", status)
