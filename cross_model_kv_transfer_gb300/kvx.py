"""ctypes binding of the kvx C ABI (``include/kvx.h``).

Argument marshalling only: the functions below have the C names and pass
device pointers straight through; every step of the transfer runs in the
CUDA kernels of ``libkvx.so``.  There is no fallback: if the library cannot
be loaded (or built with nvcc on first use), importing the symbols raises.

Low level (same names as the C ABI): ``kvx_plan_create``, ``kvx_transfer``,
``kvx_plan_destroy``, ``kvx_status_string``, ``kvx_plan_kernel``,
``kvx_plan_launches``, ``kvx_plan_cta_group``, ``kvx_transfer_static``,
``kvx_kv_diagnostics`` taking the ctypes structures ``PlanDesc`` /
``TransferArgs`` / ``DiagArgs``.

Convenience: ``Plan`` (owns a plan handle), ``Plan.transfer(...)`` which
takes torch CUDA tensors, checks their shapes, dtypes and devices, and calls
``kvx_transfer`` on the current torch stream, and ``Plan.kv_diagnostics(...)``
(fidelity statistics of a mapped cache against the target's own).  Decoding on a
transferred cache: ``Rope`` (rotary positions of new queries and keys) and
``Cache8``, one layer's 8-bit paged cache with its ``write``, ``attend`` and
``evict``; low level ``kvx_rope_init``, ``kvx_rope_apply``, ``kvx_cache8_write``,
``kvx_attend8`` and ``kvx_evict8`` with their ``*_workspace_bytes``.  Several
continuations of one prompt: ``Cache8.attend_shared`` (attention over a prefix
that requests share and their own slots), ``Pages`` (references to a pool's pages,
with ``fork``, ``reserve``, ``free`` and ``compact``), ``copy_pages`` and
``beam_select``; low level ``kvx_attend8_shared``, ``kvx_pages_*``,
``kvx_cache8_copy`` and ``kvx_beam_select``.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

from . import build as _build

# --- constants mirrored from include/kvx.h ---------------------------------
KVX_OK = 0
KVX_ERR_INVALID_ARG = 1
KVX_ERR_PAIR_MISMATCH = 2
KVX_ERR_UNSUPPORTED = 3
KVX_ERR_CUDA = 4
KVX_ERR_NO_MEMORY = 5
KVX_ERR_TOO_LARGE = 6

KVX_FLAG_BAD_LAYER_INDEX = 1
KVX_FLAG_BAD_POSITION = 2
KVX_FLAG_BAD_BLOCK = 4
KVX_FLAG_BAD_ROW = 8
KVX_FLAG_TIMEOUT = 16
KVX_FLAG_BAD_SEQLENS = 32
KVX_FLAG_BAD_SRC_BLOCK = 64
KVX_FLAG_NOT_SPD = 128
KVX_FLAG_BAD_LENGTH = 256
KVX_FLAG_NOT_FINITE = 512
KVX_FLAG_NO_PAGES = 1024

KVX_F32 = 0
KVX_BF16 = 1
KVX_CONTIGUOUS = 0
KVX_PAGED = 1
KVX_KERNEL_AUTO = 0
KVX_KERNEL_SIMT = 1
KVX_KERNEL_TCGEN05 = 2
KVX_PLAN_TEST_STALL = 1
KVX_PLAN_TC_SINGLE_CTA = 2
KVX_MAPPER_PER_HEAD = 0
KVX_MAPPER_WIDE = 1
KVX_ROPE_HALF = 0
KVX_ROPE_INTERLEAVED = 1
KVX_ROPE_UNSCALED = 0
KVX_ROPE_LINEAR = 1
KVX_ROPE_BANDS = 2
KVX_ROPE_YARN = 3

EXPORTED = ("kvx_plan_create", "kvx_transfer", "kvx_plan_destroy",
            "kvx_status_string", "kvx_plan_kernel", "kvx_plan_launches",
            "kvx_plan_cta_group", "kvx_transfer_static", "kvx_kv_diagnostics",
            "kvx_ridge_workspace_bytes", "kvx_ridge_fit",
            "kvx_layer_scores_workspace_bytes", "kvx_layer_scores",
            "kvx_rope_init", "kvx_rope_apply", "kvx_cache8_write",
            "kvx_attend8_workspace_bytes", "kvx_attend8",
            "kvx_evict8_workspace_bytes", "kvx_evict8",
            "kvx_attend8_shared_workspace_bytes", "kvx_attend8_shared",
            "kvx_pages_fork", "kvx_pages_free", "kvx_pages_reserve", "kvx_pages_compact",
            "kvx_pages_workspace_bytes", "kvx_cache8_copy",
            "kvx_beam_workspace_bytes", "kvx_beam_select")


class PlanDesc(ctypes.Structure):
    _fields_ = [
        ("src_layers", ctypes.c_int32), ("tgt_layers", ctypes.c_int32),
        ("src_kv_heads", ctypes.c_int32), ("tgt_kv_heads", ctypes.c_int32),
        ("src_head_dim", ctypes.c_int32), ("tgt_head_dim", ctypes.c_int32),
        ("k", ctypes.c_int32),
        ("rope_theta_src", ctypes.c_double), ("rope_theta_tgt", ctypes.c_double),
        ("kv_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32), ("b_dtype", ctypes.c_int32),
        ("dst_layout", ctypes.c_int32), ("block_size", ctypes.c_int32),
        ("max_position", ctypes.c_int32), ("kernel", ctypes.c_int32),
        ("tiles_per_item", ctypes.c_int32), ("flags", ctypes.c_int32),
        ("mapper", ctypes.c_int32), ("max_tokens", ctypes.c_int32),
        ("src_layout", ctypes.c_int32), ("src_block_size", ctypes.c_int32),
    ]


class TransferArgs(ctypes.Structure):
    _fields_ = [
        ("src_k", ctypes.c_void_p), ("src_v", ctypes.c_void_p),
        ("ntok", ctypes.c_int64), ("num_requests", ctypes.c_int32),
        ("cu_seqlens", ctypes.c_void_p), ("layer_idx", ctypes.c_void_p),
        ("w", ctypes.c_void_p), ("b", ctypes.c_void_p),
        ("src_pos", ctypes.c_void_p), ("tgt_pos", ctypes.c_void_p),
        ("tgt_offset", ctypes.c_void_p),
        ("dst_k", ctypes.c_void_p), ("dst_v", ctypes.c_void_p),
        ("dst_capacity", ctypes.c_int64), ("num_blocks", ctypes.c_int64),
        ("block_table", ctypes.c_void_p), ("max_blocks_per_req", ctypes.c_int32),
        ("status", ctypes.c_void_p),
        ("src_num_blocks", ctypes.c_int64), ("src_block_table", ctypes.c_void_p),
        ("max_src_blocks_per_req", ctypes.c_int32),
    ]


class DiagArgs(ctypes.Structure):
    _fields_ = [
        ("mapped_k", ctypes.c_void_p), ("mapped_v", ctypes.c_void_p),
        ("ref_k", ctypes.c_void_p), ("ref_v", ctypes.c_void_p),
        ("ntok", ctypes.c_int64), ("num_requests", ctypes.c_int32),
        ("cu_seqlens", ctypes.c_void_p),
        ("src_pos", ctypes.c_void_p), ("tgt_pos", ctypes.c_void_p),
        ("tgt_offset", ctypes.c_void_p),
        ("dst_capacity", ctypes.c_int64), ("num_blocks", ctypes.c_int64),
        ("block_table", ctypes.c_void_p), ("max_blocks_per_req", ctypes.c_int32),
        ("stats", ctypes.c_void_p), ("status", ctypes.c_void_p),
    ]


class RidgeArgs(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("n", ctypes.c_int64),
        ("p", ctypes.c_int32), ("q", ctypes.c_int32),
        ("lambda", ctypes.c_double), ("x_dtype", ctypes.c_int32),
        ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
        ("w", ctypes.c_void_p), ("b", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("status", ctypes.c_void_p),
    ]


class ScoreArgs(ctypes.Structure):
    _fields_ = [
        ("src_k", ctypes.c_void_p), ("src_v", ctypes.c_void_p),
        ("tgt_k", ctypes.c_void_p), ("tgt_v", ctypes.c_void_p),
        ("ntok", ctypes.c_int64), ("num_requests", ctypes.c_int32),
        ("cu_seqlens", ctypes.c_void_p), ("src_pos", ctypes.c_void_p),
        ("layer_idx", ctypes.c_void_p), ("lambda", ctypes.c_double),
        ("r2", ctypes.c_void_p), ("r2_set", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("status", ctypes.c_void_p),
    ]


class FeatureArgs(ctypes.Structure):
    _fields_ = [
        ("src_k", ctypes.c_void_p), ("src_v", ctypes.c_void_p),
        ("tgt_k", ctypes.c_void_p), ("tgt_v", ctypes.c_void_p),
        ("ntok", ctypes.c_int64), ("num_requests", ctypes.c_int32),
        ("cu_seqlens", ctypes.c_void_p), ("src_pos", ctypes.c_void_p),
        ("layer_idx", ctypes.c_void_p), ("out_dtype", ctypes.c_int32),
        ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
        ("status", ctypes.c_void_p),
    ]


class RopeDesc(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
        ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
        ("theta", ctypes.c_double), ("factor", ctypes.c_double),
        ("low_band", ctypes.c_double), ("high_band", ctypes.c_double),
        ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
        ("amplitude", ctypes.c_double), ("original_context", ctypes.c_int32),
    ]


class RopeState(ctypes.Structure):
    """``kvx_rope``: what ``kvx_rope_init`` fills."""
    _fields_ = [
        ("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
        ("layout", ctypes.c_int32), ("amplitude", ctypes.c_float),
        ("turns", ctypes.c_uint64 * 128),
    ]


class RopeArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
        ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p),
        ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
        ("k_token_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
        ("q_out_token_stride", ctypes.c_int64), ("q_out_head_stride", ctypes.c_int64),
        ("k_out_token_stride", ctypes.c_int64), ("k_out_head_stride", ctypes.c_int64),
        ("ntok", ctypes.c_int64), ("q_heads", ctypes.c_int32), ("k_heads", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("transpose", ctypes.c_int32),
        ("positions", ctypes.c_void_p), ("first_position", ctypes.c_int64),
        ("status", ctypes.c_void_p),
    ]


class Cache8Desc(ctypes.Structure):
    """``kvx_cache8``."""
    _fields_ = [
        ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("num_blocks", ctypes.c_int64), ("heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32),
        ("max_blocks_per_req", ctypes.c_int32), ("block_table", ctypes.c_void_p),
    ]


class Cache8WriteArgs(ctypes.Structure):
    _fields_ = [
        ("cache", Cache8Desc), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("k_token_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
        ("v_token_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("num_requests", ctypes.c_int32), ("ntok", ctypes.c_int64),
        ("cu_seqlens", ctypes.c_void_p), ("start", ctypes.c_void_p),
        ("src_rows", ctypes.c_void_p), ("num_src_rows", ctypes.c_int64),
        ("status", ctypes.c_void_p),
    ]


class Attend8Args(ctypes.Structure):
    _fields_ = [
        ("cache", Cache8Desc), ("q", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
        ("out_token_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("q_heads", ctypes.c_int32), ("ntok", ctypes.c_int64),
        ("num_requests", ctypes.c_int32), ("max_new", ctypes.c_int32),
        ("cu_seqlens", ctypes.c_void_p), ("lens", ctypes.c_void_p),
        ("max_len", ctypes.c_int32), ("scale", ctypes.c_float), ("lse", ctypes.c_void_p),
        ("weights", ctypes.c_void_p), ("weights_stride", ctypes.c_int64),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("status", ctypes.c_void_p),
    ]


class Evict8Args(ctypes.Structure):
    _fields_ = [
        ("cache", Cache8Desc), ("dst_table", ctypes.c_void_p),
        ("max_dst_blocks", ctypes.c_int32), ("num_requests", ctypes.c_int32),
        ("lens", ctypes.c_void_p), ("max_len", ctypes.c_int32), ("keep", ctypes.c_int32),
        ("sinks", ctypes.c_int32), ("recent", ctypes.c_int32),
        ("weights", ctypes.c_void_p), ("weights_stride", ctypes.c_int64),
        ("kept", ctypes.c_void_p), ("kept_weights", ctypes.c_void_p),
        ("new_lens", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t), ("status", ctypes.c_void_p),
    ]


class Attend8SharedArgs(ctypes.Structure):
    _fields_ = [
        ("own", Attend8Args), ("prefix_table", ctypes.c_void_p), ("prefix_lens", ctypes.c_void_p),
        ("groups", ctypes.c_void_p), ("max_prefix_blocks", ctypes.c_int32),
        ("num_prefixes", ctypes.c_int32), ("max_prefix", ctypes.c_int32),
        ("max_group", ctypes.c_int32),
    ]


class PagesForkArgs(ctypes.Structure):
    _fields_ = [
        ("refs", ctypes.c_void_p), ("num_blocks", ctypes.c_int64), ("block_size", ctypes.c_int32),
        ("num_rows", ctypes.c_int32), ("width", ctypes.c_int32), ("table", ctypes.c_void_p),
        ("lens", ctypes.c_void_p), ("parents", ctypes.c_void_p), ("num_new", ctypes.c_int32),
        ("new_table", ctypes.c_void_p), ("new_lens", ctypes.c_void_p), ("status", ctypes.c_void_p),
    ]


class PagesFreeArgs(ctypes.Structure):
    _fields_ = [
        ("refs", ctypes.c_void_p), ("num_blocks", ctypes.c_int64), ("num_rows", ctypes.c_int32),
        ("width", ctypes.c_int32), ("table", ctypes.c_void_p), ("status", ctypes.c_void_p),
    ]


class PagesReserveArgs(ctypes.Structure):
    _fields_ = [
        ("refs", ctypes.c_void_p), ("num_blocks", ctypes.c_int64), ("block_size", ctypes.c_int32),
        ("num_rows", ctypes.c_int32), ("width", ctypes.c_int32), ("table", ctypes.c_void_p),
        ("lens", ctypes.c_void_p), ("add", ctypes.c_void_p), ("add_all", ctypes.c_int32),
        ("copies", ctypes.c_void_p), ("caches", ctypes.c_void_p), ("num_caches", ctypes.c_int32),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("status", ctypes.c_void_p),
    ]


class PagesCompactArgs(ctypes.Structure):
    _fields_ = [
        ("refs", ctypes.c_void_p), ("num_blocks", ctypes.c_int64), ("block_size", ctypes.c_int32),
        ("tables", ctypes.c_void_p), ("entries", ctypes.c_void_p), ("num_tables", ctypes.c_int32),
        ("used", ctypes.c_void_p), ("moved", ctypes.c_void_p), ("caches", ctypes.c_void_p),
        ("num_caches", ctypes.c_int32), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t), ("status", ctypes.c_void_p),
    ]


class Cache8CopyArgs(ctypes.Structure):
    _fields_ = [
        ("caches", ctypes.c_void_p), ("num_caches", ctypes.c_int32), ("pairs", ctypes.c_void_p),
        ("num_pairs", ctypes.c_int32), ("count", ctypes.c_void_p), ("status", ctypes.c_void_p),
    ]


class BeamArgs(ctypes.Structure):
    _fields_ = [
        ("logits", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("dtype", ctypes.c_int32),
        ("num_requests", ctypes.c_int32), ("beams", ctypes.c_int32), ("out_beams", ctypes.c_int32),
        ("vocab", ctypes.c_int32), ("eos", ctypes.c_int32), ("scores", ctypes.c_void_p),
        ("done", ctypes.c_void_p), ("tokens", ctypes.c_void_p), ("parents", ctypes.c_void_p),
        ("new_scores", ctypes.c_void_p), ("new_done", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("status", ctypes.c_void_p),
    ]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def load():
    """Load ``libkvx.so`` (building it with nvcc if it is missing or stale)."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.build()
            if not os.path.exists(path):
                raise RuntimeError(f"kvx CUDA library missing: {path}")
            lib = ctypes.CDLL(path)
            lib.kvx_plan_create.argtypes = [ctypes.POINTER(PlanDesc),
                                            ctypes.POINTER(ctypes.c_void_p)]
            lib.kvx_plan_create.restype = ctypes.c_int
            lib.kvx_transfer.argtypes = [ctypes.c_void_p, ctypes.POINTER(TransferArgs),
                                         ctypes.c_void_p]
            lib.kvx_transfer.restype = ctypes.c_int
            lib.kvx_plan_destroy.argtypes = [ctypes.c_void_p]
            lib.kvx_plan_destroy.restype = ctypes.c_int
            lib.kvx_status_string.argtypes = [ctypes.c_int]
            lib.kvx_status_string.restype = ctypes.c_char_p
            lib.kvx_plan_kernel.argtypes = [ctypes.c_void_p]
            lib.kvx_plan_kernel.restype = ctypes.c_int32
            lib.kvx_plan_launches.argtypes = [ctypes.c_void_p]
            lib.kvx_plan_launches.restype = ctypes.c_int32
            lib.kvx_plan_cta_group.argtypes = [ctypes.c_void_p]
            lib.kvx_plan_cta_group.restype = ctypes.c_int32
            lib.kvx_transfer_static.argtypes = [ctypes.POINTER(PlanDesc),
                                                ctypes.POINTER(TransferArgs), ctypes.c_void_p]
            lib.kvx_transfer_static.restype = ctypes.c_int
            lib.kvx_kv_diagnostics.argtypes = [ctypes.c_void_p, ctypes.POINTER(DiagArgs),
                                               ctypes.c_void_p]
            lib.kvx_kv_diagnostics.restype = ctypes.c_int
            lib.kvx_ridge_workspace_bytes.argtypes = [ctypes.c_int32, ctypes.c_int32,
                                                      ctypes.c_int32]
            lib.kvx_ridge_workspace_bytes.restype = ctypes.c_size_t
            lib.kvx_ridge_fit.argtypes = [ctypes.POINTER(RidgeArgs), ctypes.c_void_p]
            lib.kvx_ridge_fit.restype = ctypes.c_int
            lib.kvx_layer_scores_workspace_bytes.argtypes = [ctypes.c_void_p, ctypes.c_int64]
            lib.kvx_layer_scores_workspace_bytes.restype = ctypes.c_size_t
            lib.kvx_layer_scores.argtypes = [ctypes.c_void_p, ctypes.POINTER(ScoreArgs),
                                             ctypes.c_void_p]
            lib.kvx_layer_scores.restype = ctypes.c_int
            lib.kvx_ridge_features.argtypes = [ctypes.c_void_p, ctypes.POINTER(FeatureArgs),
                                               ctypes.c_void_p]
            lib.kvx_ridge_features.restype = ctypes.c_int
            # the decoding calls take their argument block as a ctypes
            # structure (byref) or as packed bytes
            for name, argtypes in (
                    ("kvx_rope_init", [ctypes.POINTER(RopeDesc), ctypes.POINTER(RopeState)]),
                    ("kvx_rope_apply", [ctypes.c_void_p] * 3),
                    ("kvx_cache8_write", [ctypes.c_void_p] * 2),
                    ("kvx_attend8", [ctypes.c_void_p] * 2),
                    ("kvx_evict8", [ctypes.c_void_p] * 2),
                    ("kvx_attend8_shared", [ctypes.c_void_p] * 2),
                    ("kvx_pages_fork", [ctypes.c_void_p] * 2),
                    ("kvx_pages_free", [ctypes.c_void_p] * 2),
                    ("kvx_pages_reserve", [ctypes.c_void_p] * 2),
                    ("kvx_pages_compact", [ctypes.c_void_p] * 2),
                    ("kvx_cache8_copy", [ctypes.c_void_p] * 2),
                    ("kvx_beam_select", [ctypes.c_void_p] * 2)):
                getattr(lib, name).argtypes = argtypes
                getattr(lib, name).restype = ctypes.c_int
            for name in ("kvx_attend8_workspace_bytes", "kvx_evict8_workspace_bytes",
                         "kvx_attend8_shared_workspace_bytes", "kvx_beam_workspace_bytes"):
                getattr(lib, name).argtypes = [ctypes.c_void_p]
                getattr(lib, name).restype = ctypes.c_size_t
            lib.kvx_pages_workspace_bytes.argtypes = [ctypes.c_int64]
            lib.kvx_pages_workspace_bytes.restype = ctypes.c_size_t
            _lib = lib
    return _lib


def kvx_plan_create(desc: PlanDesc):
    """Returns (status, plan handle or None)."""
    h = ctypes.c_void_p()
    st = load().kvx_plan_create(ctypes.byref(desc), ctypes.byref(h))
    return st, (h.value if st == KVX_OK else None)


def kvx_transfer(plan, args: TransferArgs, stream) -> int:
    return load().kvx_transfer(plan, ctypes.byref(args), stream)


def kvx_plan_destroy(plan) -> int:
    return load().kvx_plan_destroy(plan)


def kvx_status_string(status: int) -> str:
    return load().kvx_status_string(int(status)).decode()


def kvx_plan_kernel(plan) -> int:
    return load().kvx_plan_kernel(plan)


def kvx_plan_launches(plan) -> int:
    return load().kvx_plan_launches(plan)


def kvx_plan_cta_group(plan) -> int:
    return load().kvx_plan_cta_group(plan)


def kvx_transfer_static(desc: PlanDesc, args: TransferArgs, stream) -> int:
    """Allocation-free transfer (SIMT kernel, RoPE tables in the library's
    fixed device array); for callers that may not allocate device memory."""
    return load().kvx_transfer_static(ctypes.byref(desc), ctypes.byref(args), stream)


def kvx_kv_diagnostics(plan, args: DiagArgs, stream) -> int:
    return load().kvx_kv_diagnostics(plan, ctypes.byref(args), stream)


def kvx_ridge_workspace_bytes(batch: int, p: int, q: int) -> int:
    return int(load().kvx_ridge_workspace_bytes(int(batch), int(p), int(q)))


def kvx_ridge_fit(args: RidgeArgs, stream) -> int:
    return load().kvx_ridge_fit(ctypes.byref(args), stream)


def kvx_layer_scores_workspace_bytes(plan, ntok: int) -> int:
    return load().kvx_layer_scores_workspace_bytes(plan, int(ntok))


def kvx_layer_scores(plan, args: ScoreArgs, stream) -> int:
    return load().kvx_layer_scores(plan, ctypes.byref(args), stream)


def kvx_ridge_features(plan, args: FeatureArgs, stream) -> int:
    return load().kvx_ridge_features(plan, ctypes.byref(args), stream)


def kvx_rope_init(desc: RopeDesc):
    """Returns (status, RopeState)."""
    rope = RopeState()
    return load().kvx_rope_init(ctypes.byref(desc), ctypes.byref(rope)), rope


def kvx_rope_apply(rope: RopeState, args: RopeArgs, stream) -> int:
    return load().kvx_rope_apply(ctypes.byref(rope), ctypes.byref(args), stream)


def kvx_cache8_write(args: Cache8WriteArgs, stream) -> int:
    return load().kvx_cache8_write(ctypes.byref(args), stream)


def kvx_attend8_workspace_bytes(args: Attend8Args) -> int:
    return int(load().kvx_attend8_workspace_bytes(ctypes.byref(args)))


def kvx_attend8(args: Attend8Args, stream) -> int:
    return load().kvx_attend8(ctypes.byref(args), stream)


def kvx_evict8_workspace_bytes(args: Evict8Args) -> int:
    return int(load().kvx_evict8_workspace_bytes(ctypes.byref(args)))


def kvx_evict8(args: Evict8Args, stream) -> int:
    return load().kvx_evict8(ctypes.byref(args), stream)


def kvx_attend8_shared_workspace_bytes(args: Attend8SharedArgs) -> int:
    return int(load().kvx_attend8_shared_workspace_bytes(ctypes.byref(args)))


def kvx_attend8_shared(args: Attend8SharedArgs, stream) -> int:
    return load().kvx_attend8_shared(ctypes.byref(args), stream)


def kvx_pages_fork(args: PagesForkArgs, stream) -> int:
    return load().kvx_pages_fork(ctypes.byref(args), stream)


def kvx_pages_free(args: PagesFreeArgs, stream) -> int:
    return load().kvx_pages_free(ctypes.byref(args), stream)


def kvx_pages_reserve(args: PagesReserveArgs, stream) -> int:
    return load().kvx_pages_reserve(ctypes.byref(args), stream)


def kvx_pages_compact(args: PagesCompactArgs, stream) -> int:
    return load().kvx_pages_compact(ctypes.byref(args), stream)


def kvx_pages_workspace_bytes(num_blocks: int) -> int:
    return int(load().kvx_pages_workspace_bytes(int(num_blocks)))


def kvx_cache8_copy(args: Cache8CopyArgs, stream) -> int:
    return load().kvx_cache8_copy(ctypes.byref(args), stream)


def kvx_beam_workspace_bytes(args: BeamArgs) -> int:
    return int(load().kvx_beam_workspace_bytes(ctypes.byref(args)))


def kvx_beam_select(args: BeamArgs, stream) -> int:
    return load().kvx_beam_select(ctypes.byref(args), stream)


def ridge_fit(x, y, lam: float = 0.01, w=None, b=None, workspace=None, status=None,
              stream=None):
    """Batched ridge fit of torch CUDA tensors x [batch][n][p], y
    [batch][n][q] (fp32 or bf16, or 2-D for one fit): returns fp32 (w
    [batch][p][q], b [batch][q]), enqueued on ``stream`` (default: torch's
    current stream).  Scratch is allocated here unless ``workspace`` (a
    uint8 CUDA tensor) is given."""
    import torch
    squeeze = x.dim() == 2
    if squeeze:
        x, y = x.unsqueeze(0), y.unsqueeze(0)
    if not (x.is_cuda and y.is_cuda and x.is_contiguous() and y.is_contiguous()):
        raise ValueError("x and y must be contiguous CUDA tensors")
    if x.dtype != y.dtype:
        raise ValueError("x and y must have the same dtype")
    batch, n, p = x.shape
    if tuple(y.shape[:2]) != (batch, n):
        raise ValueError("x and y must have the same batch and observation counts")
    q = y.shape[2]
    dev = x.device
    w = torch.empty((batch, p, q), dtype=torch.float32, device=dev) if w is None else w
    b = torch.empty((batch, q), dtype=torch.float32, device=dev) if b is None else b
    need = kvx_ridge_workspace_bytes(batch, p, q)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    a = RidgeArgs(int(batch), int(n), int(p), int(q), float(lam), _dtype_code(x.dtype),
                  x.data_ptr(), y.data_ptr(), w.data_ptr(), b.data_ptr(), workspace.data_ptr(),
                  workspace.numel(), None if status is None else status.data_ptr())
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    st = kvx_ridge_fit(a, ctypes.c_void_p(stream.cuda_stream))
    if st != KVX_OK:
        raise KvxError(st, "kvx_ridge_fit")
    return (w[0], b[0]) if squeeze else (w, b)


class KvxError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {kvx_status_string(status)} (status {status})")
        self.status = status


def _dtype_code(dt) -> int:
    import torch
    if dt == torch.float32:
        return KVX_F32
    if dt == torch.bfloat16:
        return KVX_BF16
    raise ValueError(f"unsupported dtype {dt}")


class Plan:
    """A kvx plan for one (source, target) model pair on the current device."""

    def __init__(self, *, src_layers, tgt_layers, kv_heads, head_dim, k, rope_theta_src,
                 rope_theta_tgt, max_position, kv_dtype, w_dtype, b_dtype,
                 layout=KVX_CONTIGUOUS, block_size=0, kernel=KVX_KERNEL_AUTO,
                 tgt_kv_heads=None, tgt_head_dim=None, tiles_per_item=0, flags=0,
                 mapper=KVX_MAPPER_PER_HEAD, max_tokens=0, src_layout=KVX_CONTIGUOUS,
                 src_block_size=0):
        self.desc = PlanDesc(
            src_layers, tgt_layers, kv_heads,
            kv_heads if tgt_kv_heads is None else tgt_kv_heads,
            head_dim, head_dim if tgt_head_dim is None else tgt_head_dim, k,
            float(rope_theta_src), float(rope_theta_tgt),
            _dtype_code(kv_dtype), _dtype_code(w_dtype), _dtype_code(b_dtype),
            int(layout), int(block_size), int(max_position), int(kernel),
            int(tiles_per_item), int(flags), int(mapper), int(max_tokens), int(src_layout),
            int(src_block_size))
        self.kv_dtype, self.w_dtype, self.b_dtype = kv_dtype, w_dtype, b_dtype
        st, h = kvx_plan_create(self.desc)
        if st != KVX_OK:
            raise KvxError(st, "kvx_plan_create")
        self.handle = h

    @property
    def kernel(self) -> int:
        return kvx_plan_kernel(self.handle)

    @property
    def cta_group(self) -> int:
        return kvx_plan_cta_group(self.handle)

    @property
    def launches_per_transfer(self) -> int:
        return kvx_plan_launches(self.handle)

    def close(self):
        if getattr(self, "handle", None):
            kvx_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def make_args(self, *, src_k, src_v, layer_idx, w, b, dst_k, dst_v, cu_seqlens=None,
                  src_pos=None, tgt_pos=None, tgt_offset=None,
                  dst_capacity=None, num_blocks=None, block_table=None,
                  status=None, ntok=None, src_block_table=None) -> TransferArgs:
        """Check tensors against the plan and pack a ``TransferArgs``.  A
        paged source ([Ls][src_num_blocks*src_block_size][H][d]) needs
        ``src_block_table`` [R][max] and ``ntok`` (the packed token count)."""
        import torch
        d = self.desc
        Ls, Lt, H, hd, k = d.src_layers, d.tgt_layers, d.src_kv_heads, d.src_head_dim, d.k

        def ptr(t, name, dtype, shape=None, ndim=None):
            if t is None:
                return None
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            if t.dtype != dtype:
                raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            if shape is not None and tuple(t.shape) != tuple(shape):
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
            if ndim is not None and t.dim() != ndim:
                raise ValueError(f"{name} must have {ndim} dims")
            return t.data_ptr()

        R = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
        a = TransferArgs()
        if d.src_layout == KVX_PAGED:
            if ntok is None or src_block_table is None:
                raise ValueError("a paged source needs ntok and src_block_table")
            src_rows = src_k.shape[1]
            if src_rows % d.src_block_size:
                raise ValueError("source rows must be whole blocks")
            a.src_num_blocks = src_rows // d.src_block_size
            a.src_block_table = ptr(src_block_table, "src_block_table", torch.int32, ndim=2)
            a.max_src_blocks_per_req = int(src_block_table.shape[1])
        else:
            ntok = src_k.shape[1] if ntok is None else int(ntok)
            src_rows = ntok
        a.src_k = ptr(src_k, "src_k", self.kv_dtype, (Ls, src_rows, H, hd))
        a.src_v = ptr(src_v, "src_v", self.kv_dtype, (Ls, src_rows, H, hd))
        a.ntok = ntok
        a.num_requests = R
        a.cu_seqlens = ptr(cu_seqlens, "cu_seqlens", torch.int32, (R + 1,))
        a.layer_idx = ptr(layer_idx, "layer_idx", torch.int32, (Lt, k))
        if d.mapper == KVX_MAPPER_WIDE:
            a.w = ptr(w, "w", self.w_dtype, (Lt, k * 2 * H * hd, H * 2 * hd))
        else:
            a.w = ptr(w, "w", self.w_dtype, (Lt, H, 2, k * hd, hd))
        a.b = ptr(b, "b", self.b_dtype, (Lt, H, 2, hd))
        a.src_pos = ptr(src_pos, "src_pos", torch.int32, (ntok,))
        a.tgt_pos = ptr(tgt_pos, "tgt_pos", torch.int32, (ntok,))
        a.tgt_offset = ptr(tgt_offset, "tgt_offset", torch.int32, (R,))
        if d.dst_layout == KVX_CONTIGUOUS:
            cap = int(dst_capacity) if dst_capacity is not None else dst_k.shape[1] // R
            rows = R * cap
            a.dst_capacity = cap
        else:
            nb = int(num_blocks) if num_blocks is not None else dst_k.shape[1] // d.block_size
            rows = nb * d.block_size
            a.num_blocks = nb
            a.block_table = ptr(block_table, "block_table", torch.int32, ndim=2)
            a.max_blocks_per_req = int(block_table.shape[1])
        a.dst_k = ptr(dst_k, "dst_k", self.kv_dtype, (Lt, rows, H, hd))
        a.dst_v = ptr(dst_v, "dst_v", self.kv_dtype, (Lt, rows, H, hd))
        a.status = ptr(status, "status", torch.int32, (1,))
        a._keep = (src_k, src_v, cu_seqlens, layer_idx, w, b, src_pos, tgt_pos, tgt_offset,
                   dst_k, dst_v, block_table, status, src_block_table)
        return a

    def transfer(self, stream=None, **tensors) -> None:
        """Enqueue one transfer on ``stream`` (default: torch's current stream)."""
        import torch
        args = self.make_args(**tensors)
        if stream is None:
            stream = torch.cuda.current_stream()
        st = kvx_transfer(self.handle, args, ctypes.c_void_p(stream.cuda_stream))
        if st != KVX_OK:
            raise KvxError(st, "kvx_transfer")

    def make_diag_args(self, *, mapped_k, mapped_v, ref_k, ref_v, stats, ntok, cu_seqlens=None,
                       src_pos=None, tgt_pos=None, tgt_offset=None, dst_capacity=None,
                       num_blocks=None, block_table=None, status=None) -> DiagArgs:
        """Check tensors against the plan and pack a ``DiagArgs``."""
        import torch
        d = self.desc
        Lt, H, hd = d.tgt_layers, d.tgt_kv_heads, d.tgt_head_dim
        R = 1 if cu_seqlens is None else cu_seqlens.numel() - 1

        def ptr(t, name, dtype, shape=None, ndim=None):
            if t is None:
                return None
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            if t.dtype != dtype:
                raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            if shape is not None and tuple(t.shape) != tuple(shape):
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
            if ndim is not None and t.dim() != ndim:
                raise ValueError(f"{name} must have {ndim} dims")
            return t.data_ptr()

        a = DiagArgs()
        a.ntok = int(ntok)
        a.num_requests = R
        a.cu_seqlens = ptr(cu_seqlens, "cu_seqlens", torch.int32, (R + 1,))
        a.src_pos = ptr(src_pos, "src_pos", torch.int32, (int(ntok),))
        a.tgt_pos = ptr(tgt_pos, "tgt_pos", torch.int32, (int(ntok),))
        a.tgt_offset = ptr(tgt_offset, "tgt_offset", torch.int32, (R,))
        if d.dst_layout == KVX_CONTIGUOUS:
            cap = int(dst_capacity) if dst_capacity is not None else ref_k.shape[1] // R
            rows = R * cap
            a.dst_capacity = cap
        else:
            nb = int(num_blocks) if num_blocks is not None else ref_k.shape[1] // d.block_size
            rows = nb * d.block_size
            a.num_blocks = nb
            a.block_table = ptr(block_table, "block_table", torch.int32, ndim=2)
            a.max_blocks_per_req = int(block_table.shape[1])
        shape = (Lt, rows, H, hd)
        a.mapped_k = ptr(mapped_k, "mapped_k", self.kv_dtype, shape)
        a.mapped_v = ptr(mapped_v, "mapped_v", self.kv_dtype, shape)
        a.ref_k = ptr(ref_k, "ref_k", self.kv_dtype, shape)
        a.ref_v = ptr(ref_v, "ref_v", self.kv_dtype, shape)
        a.stats = ptr(stats, "stats", torch.float64, (Lt, H, 2, hd + 4))
        a.status = ptr(status, "status", torch.int32, (1,))
        a._keep = (mapped_k, mapped_v, ref_k, ref_v, stats, cu_seqlens, src_pos, tgt_pos,
                   tgt_offset, block_table, status)
        return a

    def layer_scores(self, *, src_k, src_v, tgt_k, tgt_v, lam=0.01, cu_seqlens=None,
                     src_pos=None, layer_idx=None, r2=None, r2_set=None, workspace=None,
                     status=None, stream=None):
        """Layer-selection scores (``kvx_layer_scores``) of CUDA tensors:
        src_k / src_v [Ls][ntok][H][d] and tgt_k / tgt_v [Lt][ntok][H][d] of
        the same tokens; returns fp64 r2 [Lt][Ls][H][2] and, with
        ``layer_idx`` [Lt][k], r2_set [Lt][H][2] (else None), enqueued on
        ``stream``.  Scratch is allocated here unless ``workspace`` (a uint8
        CUDA tensor) is given."""
        import torch
        d = self.desc
        Ls, Lt, H, hd = d.src_layers, d.tgt_layers, d.src_kv_heads, d.src_head_dim
        for name, t, L in (("src_k", src_k, Ls), ("src_v", src_v, Ls), ("tgt_k", tgt_k, Lt),
                           ("tgt_v", tgt_v, Lt)):
            if not (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous CUDA tensor")
            if t.dtype != self.kv_dtype or t.dim() != 4 or t.shape[0] != L or \
                    tuple(t.shape[2:]) != (H, hd):
                raise ValueError(f"{name}: expected [{L}][ntok][{H}][{hd}] {self.kv_dtype}")
        ntok = src_k.shape[1]
        if any(t.shape[1] != ntok for t in (src_v, tgt_k, tgt_v)):
            raise ValueError("the four caches must hold the same tokens")
        dev = src_k.device
        R = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
        r2 = torch.empty((Lt, Ls, H, 2), dtype=torch.float64, device=dev) if r2 is None else r2
        if layer_idx is not None and r2_set is None:
            r2_set = torch.empty((Lt, H, 2), dtype=torch.float64, device=dev)
        need = kvx_layer_scores_workspace_bytes(self.handle, ntok)
        if need == 0:
            raise KvxError(KVX_ERR_UNSUPPORTED, "kvx_layer_scores_workspace_bytes")
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        ptr = lambda t: None if t is None else t.data_ptr()
        for name, t, shape in (("cu_seqlens", cu_seqlens, (R + 1,)), ("src_pos", src_pos, (ntok,)),
                               ("layer_idx", layer_idx, (Lt, d.k))):
            if t is not None and (t.dtype != torch.int32 or tuple(t.shape) != shape or
                                  not t.is_cuda or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous int32 CUDA tensor {shape}")
        a = ScoreArgs(src_k.data_ptr(), src_v.data_ptr(), tgt_k.data_ptr(), tgt_v.data_ptr(),
                      int(ntok), int(R), ptr(cu_seqlens), ptr(src_pos), ptr(layer_idx),
                      float(lam), r2.data_ptr(), ptr(r2_set), workspace.data_ptr(),
                      workspace.numel(), ptr(status))
        if stream is None:
            stream = torch.cuda.current_stream(dev)
        st = kvx_layer_scores(self.handle, a, ctypes.c_void_p(stream.cuda_stream))
        if st != KVX_OK:
            raise KvxError(st, "kvx_layer_scores")
        return r2, r2_set

    def ridge_features(self, *, src_k, src_v, layer_idx, tgt_k=None, tgt_v=None,
                       cu_seqlens=None, src_pos=None, out_dtype=None, x=None, y=None,
                       status=None, stream=None):
        """Content-space observations of the maps' ridge fits
        (``kvx_ridge_features``) from CUDA caches src_k / src_v
        [Ls][ntok][H][d] and, for y, tgt_k / tgt_v [Lt][ntok][H][d] of the
        same tokens: returns x [Lt*H*2][ntok][k*d] and y [Lt*H*2][ntok][d]
        (None without the target caches) in ``out_dtype`` (default fp32),
        enqueued on ``stream`` -- the x and y of one ``ridge_fit`` whose W
        and b this plan's transfer reads."""
        import torch
        d = self.desc
        Ls, Lt, H, hd, k = d.src_layers, d.tgt_layers, d.src_kv_heads, d.src_head_dim, d.k
        if layer_idx is None:
            raise ValueError("layer_idx [Lt][k] is required")
        with_y = tgt_k is not None or tgt_v is not None
        caches = [("src_k", src_k, Ls), ("src_v", src_v, Ls)]
        if with_y:
            caches += [("tgt_k", tgt_k, Lt), ("tgt_v", tgt_v, Lt)]
        for name, t, L in caches:
            if not (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous CUDA tensor")
            if t.dtype != self.kv_dtype or t.dim() != 4 or t.shape[0] != L or \
                    tuple(t.shape[2:]) != (H, hd):
                raise ValueError(f"{name}: expected [{L}][ntok][{H}][{hd}] {self.kv_dtype}")
        ntok = src_k.shape[1]
        if any(t.shape[1] != ntok for _, t, _ in caches):
            raise ValueError("the caches must hold the same tokens")
        R = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
        for name, t, shape in (("cu_seqlens", cu_seqlens, (R + 1,)), ("src_pos", src_pos, (ntok,)),
                               ("layer_idx", layer_idx, (Lt, k))):
            if t is not None and (t.dtype != torch.int32 or tuple(t.shape) != shape or
                                  not t.is_cuda or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous int32 CUDA tensor {shape}")
        out_dtype = torch.float32 if out_dtype is None else out_dtype
        dev = src_k.device
        B = Lt * H * 2
        for name, t, shape in (("x", x, (B, ntok, k * hd)), ("y", y, (B, ntok, hd))):
            if t is not None and (t.dtype != out_dtype or tuple(t.shape) != shape or
                                  not t.is_cuda or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous {out_dtype} CUDA tensor {shape}")
        if x is None:
            x = torch.empty((B, ntok, k * hd), dtype=out_dtype, device=dev)
        if with_y and y is None:
            y = torch.empty((B, ntok, hd), dtype=out_dtype, device=dev)
        ptr = lambda t: None if t is None else t.data_ptr()
        a = FeatureArgs(src_k.data_ptr(), src_v.data_ptr(), ptr(tgt_k), ptr(tgt_v), int(ntok),
                        int(R), ptr(cu_seqlens), ptr(src_pos), layer_idx.data_ptr(),
                        _dtype_code(out_dtype), x.data_ptr(), ptr(y if with_y else None),
                        ptr(status))
        if stream is None:
            stream = torch.cuda.current_stream(dev)
        st = kvx_ridge_features(self.handle, a, ctypes.c_void_p(stream.cuda_stream))
        if st != KVX_OK:
            raise KvxError(st, "kvx_ridge_features")
        return x, (y if with_y else None)

    def kv_diagnostics(self, stream=None, **tensors) -> None:
        """Enqueue the fidelity statistics [Lt][H][2][d + 4] (fp64, into
        ``stats``) of a mapped cache against the target's own cache on
        ``stream`` (default: torch's current stream)."""
        import torch
        args = self.make_diag_args(**tensors)
        if stream is None:
            stream = torch.cuda.current_stream()
        st = kvx_kv_diagnostics(self.handle, args, ctypes.c_void_p(stream.cuda_stream))
        if st != KVX_OK:
            raise KvxError(st, "kvx_kv_diagnostics")


# --- decoding on a transferred cache -----------------------------------------

def _packer(cls):
    """``struct`` packer of a ctypes structure's fields (nested ones in line,
    native alignment): one pack is several times cheaper than as many
    attribute stores, which is what a single-token call spends its time on."""
    letters = {ctypes.c_void_p: "P", ctypes.c_int32: "i", ctypes.c_int64: "q",
               ctypes.c_float: "f", ctypes.c_size_t: "N"}

    def fmt(c):
        return "".join(fmt(t) if issubclass(t, ctypes.Structure) else letters[t]
                       for _, t in c._fields_)

    s = struct.Struct("@" + fmt(cls))
    assert s.size <= ctypes.sizeof(cls) < s.size + 8
    return s.pack


_WORKSPACE_HEAD = 1024    # bytes of a kvx_attend8 workspace that must be zero at first
_pack_rope = _packer(RopeArgs)
_pack_write = _packer(Cache8WriteArgs)
_pack_attend = _packer(Attend8Args)
_pack_evict = _packer(Evict8Args)
_pack_shared = _packer(Attend8SharedArgs)
_pack_cache = _packer(Cache8Desc)
_pack_fork = _packer(PagesForkArgs)
_pack_reserve = _packer(PagesReserveArgs)
_pack_compact = _packer(PagesCompactArgs)
_pack_beam = _packer(BeamArgs)


class _Fast:
    """What a single-token call looks up every time, looked up once: torch, the
    library's entry points, and torch's own (device, raw stream) queries."""
    torch = None

    @classmethod
    def ready(cls):
        import torch
        lib = load()
        cls.f32, cls.bf16, cls.i32 = torch.float32, torch.bfloat16, torch.int32
        cls.codes = {torch.float32: KVX_F32, torch.bfloat16: KVX_BF16}
        cls.rope, cls.write = lib.kvx_rope_apply, lib.kvx_cache8_write
        cls.attend, cls.evict = lib.kvx_attend8, lib.kvx_evict8
        cls.shared, cls.fork = lib.kvx_attend8_shared, lib.kvx_pages_fork
        cls.reserve, cls.beam = lib.kvx_pages_reserve, lib.kvx_beam_select
        cls.compact = lib.kvx_pages_compact
        cls.empty = torch.empty
        cls.device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        cls.raw = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda i: torch.cuda.current_stream(i).cuda_stream)
        cls.torch = torch


def _int_table(t, name, device, ndim=1):
    """Data pointer of a contiguous int32 CUDA tensor (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not _Fast.i32 or t.device != device or t.dim() != ndim or \
            not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-D int32 tensor on {device}")
    return t.data_ptr()


def _workspace(t, device):
    """Pointer and bytes of a workspace: any contiguous tensor on the device."""
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return t.data_ptr(), t.numel() * t.element_size()


def _status_ptr(t, device):
    return 0 if t is None else _int_table(t, "status", device)


def _on_device(device):
    if device.type != "cuda":
        raise ValueError(f"tensors are on {device}, which is not a CUDA device")
    if _Fast.torch is None:
        _Fast.ready()
    if _Fast.device() != device.index:
        raise ValueError(f"tensors are on {device}, which is not the current CUDA device")


def _raw_stream(stream, device):
    return _Fast.raw(device.index) if stream is None else stream.cuda_stream


def _heads(t, name, dtype, device, heads, dim):
    """Check a [tokens][heads][dim] tensor with unit stride inside a head;
    returns its strides and token count."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or t.dtype is not dtype or t.device != device or shape[1] != heads or \
            shape[2] != dim or stride[2] != 1:
        raise ValueError(f"{name}: expected [tokens][{heads}][{dim}] {dtype} on {device} with "
                         f"unit stride inside a head")
    return stride, shape[0]


def _code_of(dtype):
    code = _Fast.codes.get(dtype)
    return _dtype_code(dtype) if code is None else code


class Rope:
    """A rotation of head vectors by position (``kvx_rope``).

    ``layout`` "half" pairs (i, i + rot_dim/2), "interleaved" (2i, 2i + 1);
    ``scaling`` None, "linear" (``factor``), "bands" (``factor``, ``low_band``,
    ``high_band``, ``original_context``) or "yarn" (``factor``, ``beta_fast``,
    ``beta_slow``, ``original_context``); ``amplitude`` 0 is the scaling's own.
    """

    def __init__(self, head_dim, theta, *, rot_dim=None, layout="half", scaling=None, factor=1.0,
                 low_band=0.0, high_band=0.0, beta_fast=32.0, beta_slow=1.0,
                 original_context=0, amplitude=0.0):
        layouts = {"half": KVX_ROPE_HALF, "interleaved": KVX_ROPE_INTERLEAVED}
        scalings = {None: KVX_ROPE_UNSCALED, "linear": KVX_ROPE_LINEAR, "bands": KVX_ROPE_BANDS,
                    "yarn": KVX_ROPE_YARN}
        if layout not in layouts or scaling not in scalings:
            raise ValueError(f"unknown layout {layout!r} or scaling {scaling!r}")
        desc = RopeDesc(int(head_dim), int(head_dim if rot_dim is None else rot_dim),
                        layouts[layout], scalings[scaling], float(theta), float(factor),
                        float(low_band), float(high_band), float(beta_fast), float(beta_slow),
                        float(amplitude), int(original_context))
        st, self.state = kvx_rope_init(desc)
        if st != KVX_OK:
            raise KvxError(st, "kvx_rope_init")
        self.head_dim = int(head_dim)
        self._ptr = ctypes.addressof(self.state)

    def apply(self, q=None, k=None, positions=None, *, transpose=False, first_position=0,
              q_out=None, k_out=None, status=None, stream=None):
        """Rotate q [tokens][q_heads][d] and k [tokens][k_heads][d] (either may
        be None; fp32 or bf16, any token and head strides) at ``positions``
        (int32, or first_position, first_position + 1, ...); returns (q_out,
        k_out), allocated unless given (in place with ``q_out=q``).
        ``transpose`` applies the transposed rotation: the gradient."""
        x = q if q is not None else k
        if x is None:
            raise ValueError("q or k is needed")
        dev, dt, d = x.device, x.dtype, self.head_dim
        _on_device(dev)
        code = _code_of(dt)
        n = x.shape[0]
        qp = kp = qo = ko = hq = hk = 0
        qs = ks = qos = kos = (0, 0, 0)
        if q is not None:
            hq = q.shape[1]
            qs, n = _heads(q, "q", dt, dev, hq, d)
            if q_out is None:
                q_out = _new(stream, (n, hq, d), dt, dev)
                qos = (hq * d, d, 1)
            else:
                qos, m = _heads(q_out, "q_out", dt, dev, hq, d)
                if m != n:
                    raise ValueError("q_out has another number of tokens")
            qp, qo = q.data_ptr(), q_out.data_ptr()
        if k is not None:
            hk = k.shape[1]
            ks, m = _heads(k, "k", dt, dev, hk, d)
            if m != n:
                raise ValueError("q and k must hold the same tokens")
            if k_out is None:
                k_out = _new(stream, (n, hk, d), dt, dev)
                kos = (hk * d, d, 1)
            else:
                kos, m = _heads(k_out, "k_out", dt, dev, hk, d)
                if m != n:
                    raise ValueError("k_out has another number of tokens")
            kp, ko = k.data_ptr(), k_out.data_ptr()
        pos = _int_table(positions, "positions", dev)
        if pos and positions.shape[0] != n:
            raise ValueError("positions must hold one entry for each token")
        a = _pack_rope(qp, kp, qo, ko, qs[0], qs[1], ks[0], ks[1], qos[0], qos[1], kos[0], kos[1],
                       n, hq, hk, code, 1 if transpose else 0, pos, first_position,
                       _status_ptr(status, dev))
        st = _Fast.rope(self._ptr, a, _raw_stream(stream, dev))
        if st != KVX_OK:
            raise KvxError(st, "kvx_rope_apply")
        return (None if q is None else q_out), (None if k is None else k_out)


class Cache8:
    """An 8-bit paged cache of one layer (``kvx_cache8``): e4m3 codes
    [num_blocks][heads][block_size][head_dim] (uint8 or float8_e4m3fn) and one
    fp32 scale for each (block, head), for keys and for values.  The tensors
    stay the caller's; ``Cache8.empty`` allocates them."""

    def __init__(self, k_codes, v_codes, k_scale, v_scale):
        import torch
        dev = k_codes.device
        for name, t in (("k_codes", k_codes), ("v_codes", v_codes)):
            if t.dim() != 4 or t.dtype not in (torch.uint8, torch.float8_e4m3fn) or \
                    t.shape != k_codes.shape or t.device != dev or not t.is_contiguous():
                raise ValueError(f"{name}: expected a contiguous [num_blocks][heads][block_size]"
                                 f"[head_dim] uint8 or float8_e4m3fn tensor on {dev}")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t.dtype != torch.float32 or t.shape != k_codes.shape[:2] or t.device != dev or \
                    not t.is_contiguous():
                raise ValueError(f"{name}: expected a contiguous fp32 [num_blocks][heads] tensor "
                                 f"on {dev}")
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.device = dev
        self.num_blocks, self.heads, self.block_size, self.head_dim = k_codes.shape
        self._head = (k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(),
                      v_scale.data_ptr(), self.num_blocks, self.heads, self.head_dim,
                      self.block_size)
        # as one of an array of caches, whose block tables are not used: any aligned address
        self._packed = _pack_cache(*self._head, 1, self._head[2])

    @classmethod
    def empty(cls, num_blocks, heads, head_dim, block_size, device="cuda"):
        import torch
        codes = torch.zeros((2, num_blocks, heads, block_size, head_dim), dtype=torch.uint8,
                            device=device)
        scale = torch.ones((2, num_blocks, heads), dtype=torch.float32, device=device)
        return cls(codes[0], codes[1], scale[0], scale[1])

    def _table(self, block_table):
        ptr = _int_table(block_table, "block_table", self.device, 2)
        return self._head + (block_table.shape[1], ptr)

    def write(self, k, v, block_table, start=None, *, cu_seqlens=None, src_rows=None, status=None,
              stream=None):
        """Quantise new (rotated) keys and values [tokens][heads][d] of R
        requests into their blocks: request r's tokens go to slots start[r],
        start[r] + 1, ... (0 without ``start``).  Without ``cu_seqlens`` [R + 1]
        there is one token for each request.  With ``src_rows`` token g is row
        src_rows[g] of k and v, so a paged bf16 / fp32 cache can be read."""
        dev = self.device
        _on_device(dev)
        dt = k.dtype
        ks, rows = _heads(k, "k", dt, dev, self.heads, self.head_dim)
        vs, m = _heads(v, "v", dt, dev, self.heads, self.head_dim)
        if m != rows:
            raise ValueError("k and v must hold the same rows")
        table = self._table(block_table)
        R = block_table.shape[0]
        if cu_seqlens is not None and cu_seqlens.shape[0] != R + 1:
            raise ValueError("cu_seqlens must have one entry more than block_table has rows")
        if start is not None and start.shape[0] != R:
            raise ValueError("start must hold one entry for each request")
        a = _pack_write(*table, k.data_ptr(), v.data_ptr(), ks[0], ks[1], vs[0], vs[1],
                        _code_of(dt), R, rows if src_rows is None else src_rows.shape[0],
                        _int_table(cu_seqlens, "cu_seqlens", dev),
                        _int_table(start, "start", dev), _int_table(src_rows, "src_rows", dev),
                        rows, _status_ptr(status, dev))
        st = _Fast.write(a, _raw_stream(stream, dev))
        if st != KVX_OK:
            raise KvxError(st, "kvx_cache8_write")

    def attend_workspace(self, *, ntok, num_requests, q_heads, max_len, max_new=1, dtype=None,
                         weights=False):
        """A workspace (uint8) for ``attend`` calls of at most these sizes and
        queries of ``dtype`` (bf16) that are ordered on one stream.  With
        ``weights`` it has room for scores, up to 4 GB by ``max_len``; without,
        calls with weights run in it too and form their scores a second time."""
        import torch
        return self._attend_scratch(torch.bfloat16 if dtype is None else dtype, ntok, num_requests, q_heads,
                                    max_len, max_new, weights, None)

    def _attend_scratch(self, dtype, ntok, num_requests, q_heads, max_len, max_new, weights, most_scores):
        """A workspace, with room for scores unless that takes more than ``most_scores`` bytes."""
        import torch
        a = Attend8Args()
        a.cache = Cache8Desc(*self._head, 1, self.k_codes.data_ptr())
        a.dtype = _dtype_code(dtype)
        a.q_heads, a.ntok, a.num_requests = q_heads, ntok, num_requests
        a.max_new, a.max_len, a.scale = max_new, max_len, 1.0
        a.lens = a.cu_seqlens = self.k_codes.data_ptr()   # sizes only: never read
        need = kvx_attend8_workspace_bytes(a)
        if weights:
            a.weights, a.weights_stride = self.k_scale.data_ptr(), max_len
            roomy = kvx_attend8_workspace_bytes(a)
            if roomy == 0 or most_scores is None or roomy - need <= most_scores:
                need = roomy
        if need == 0:
            raise KvxError(KVX_ERR_INVALID_ARG, "kvx_attend8_workspace_bytes")
        ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        ws[:_WORKSPACE_HEAD].zero_()
        return ws

    def attend(self, q, block_table, lens, max_len, *, cu_seqlens=None, max_new=1, scale=None,
               out=None, lse=None, weights=None, workspace=None, status=None, stream=None):
        """Attention of the new queries q [tokens][q_heads][d] over the slots
        of their requests (``lens`` [R], at most ``max_len``): query i of n sees
        slots up to lens - n + i.  With ``cu_seqlens`` [R + 1] a request has up
        to ``max_new`` queries (more: nothing is written, and ``status`` tells).
        Returns (out, lse [tokens][q_heads]); ``out`` may be q without weights.
        ``weights`` [R][heads][>= max_len] fp32 accumulates the attention weight
        of each slot.  Scratch (for scores at most 1 GB) is allocated here unless ``workspace`` (from
        ``attend_workspace``) is given."""
        dev, dt = self.device, q.dtype
        _on_device(dev)
        if q.dim() != 3:
            raise ValueError("q must be [tokens][q_heads][d]")
        hq, d = q.shape[1], self.head_dim
        qs, n = _heads(q, "q", dt, dev, hq, d)
        table = self._table(block_table)
        R = block_table.shape[0]
        if lens.shape[0] != R or (cu_seqlens is not None and cu_seqlens.shape[0] != R + 1):
            raise ValueError("lens, cu_seqlens and block_table must hold the same requests")
        code = _code_of(dt)
        out, os_, lse = self._attend_outputs(out, lse, n, hq, dt, stream)
        wptr = wstride = 0
        if weights is not None:
            wptr, wstride = self._weights(weights, R)
        if workspace is None:
            workspace = _on_stream(self._attend_scratch, stream, dt, n, R, hq, max_len, max_new,
                                   weights is not None, 1 << 30)
        a = _pack_attend(*table, q.data_ptr(), out.data_ptr(), qs[0], qs[1], os_[0], os_[1], code,
                         hq, n, R, max_new, _int_table(cu_seqlens, "cu_seqlens", dev),
                         _int_table(lens, "lens", dev), max_len,
                         d ** -0.5 if scale is None else scale, lse.data_ptr(), wptr, wstride,
                         *_workspace(workspace, dev), _status_ptr(status, dev))
        st = _Fast.attend(a, _raw_stream(stream, dev))
        if st != KVX_OK:
            raise KvxError(st, "kvx_attend8")
        return out, lse

    def _attend_outputs(self, out, lse, n, hq, dt, stream):
        """The outputs of n queries, checked or allocated, and the strides of the first."""
        dev, d = self.device, self.head_dim
        if out is None:
            out = _new(stream, (n, hq, d), dt, dev)
            os_ = (hq * d, d, 1)
        else:
            os_, m = _heads(out, "out", dt, dev, hq, d)
            if m != n:
                raise ValueError("out has another number of tokens")
        if lse is None:
            lse = _new(stream, (n, hq), _Fast.f32, dev)
        elif lse.dtype is not _Fast.f32 or tuple(lse.shape) != (n, hq) or lse.device != dev or \
                not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous fp32 [{n}][{hq}] tensor on {dev}")
        return out, os_, lse

    def attend_shared_workspace(self, *, ntok, num_requests, q_heads, max_prefix, max_len,
                                num_prefixes=1, max_group=None, max_new=1, dtype=None):
        """A workspace (uint8) for ``attend_shared`` calls of at most these sizes
        and queries of ``dtype`` (bf16) that are ordered on one stream."""
        import torch
        a = Attend8SharedArgs()
        own, any_ptr = a.own, self.k_codes.data_ptr()     # sizes only: never read
        own.cache = Cache8Desc(*self._head, 1, any_ptr)
        own.dtype = _dtype_code(torch.bfloat16 if dtype is None else dtype)
        own.q_heads, own.ntok, own.num_requests = q_heads, ntok, num_requests
        own.max_new, own.max_len, own.scale = max_new, max_len, 1.0
        own.lens = own.cu_seqlens = a.prefix_table = a.prefix_lens = a.groups = any_ptr
        a.max_prefix_blocks, a.num_prefixes, a.max_prefix = 1, num_prefixes, max_prefix
        a.max_group = num_requests if max_group is None else max_group
        need = kvx_attend8_shared_workspace_bytes(a)
        if need == 0:
            raise KvxError(KVX_ERR_INVALID_ARG, "kvx_attend8_shared_workspace_bytes")
        ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        ws[:_WORKSPACE_HEAD].zero_()
        return ws

    def attend_shared(self, q, prefix_table, prefix_lens, block_table, lens, *, max_prefix, max_len,
                      groups=None, max_group=None, cu_seqlens=None, max_new=1, scale=None, out=None,
                      lse=None, workspace=None, status=None, stream=None):
        """Attention of requests that share prefixes: as ``attend`` of sequences
        that hold a prefix's slots and then the request's own.  Requests
        groups[p] .. groups[p + 1] - 1 (``groups`` [P + 1]; without it all) have
        the slots of row p of ``prefix_table`` (``prefix_lens`` [P], at most
        ``max_prefix``) before those of ``block_table`` and ``lens``; a prefix has
        at most ``max_group`` requests (with more than max_group * max_new queries
        nothing is written, and ``status`` tells).  The new queries are the last of
        a request's own slots.  A prefix is read once for 8 to 256 rows of a
        KV head and its group.  Returns (out, lse [tokens][q_heads]) over both.
        Scratch is allocated here unless ``workspace`` (from
        ``attend_shared_workspace``) is given."""
        dev, dt = self.device, q.dtype
        _on_device(dev)
        if q.dim() != 3:
            raise ValueError("q must be [tokens][q_heads][d]")
        hq, d = q.shape[1], self.head_dim
        qs, n = _heads(q, "q", dt, dev, hq, d)
        table = self._table(block_table)
        R, P = block_table.shape[0], prefix_lens.shape[0]
        if lens.shape[0] != R or (cu_seqlens is not None and cu_seqlens.shape[0] != R + 1):
            raise ValueError("lens, cu_seqlens and block_table must hold the same requests")
        before = _int_table(prefix_table, "prefix_table", dev, 2)
        if prefix_table.shape[0] != P or (P != 1 if groups is None else groups.shape[0] != P + 1):
            raise ValueError("prefix_table, prefix_lens and groups must hold the same prefixes")
        code = _code_of(dt)
        out, os_, lse = self._attend_outputs(out, lse, n, hq, dt, stream)
        if max_group is None:
            max_group = R
        if workspace is None:
            workspace = _on_stream(self.attend_shared_workspace, stream, ntok=n, num_requests=R,
                                   q_heads=hq, max_prefix=max_prefix, max_len=max_len,
                                   num_prefixes=P, max_group=max_group, max_new=max_new, dtype=dt)
        a = _pack_shared(*table, q.data_ptr(), out.data_ptr(), qs[0], qs[1], os_[0], os_[1], code,
                         hq, n, R, max_new, _int_table(cu_seqlens, "cu_seqlens", dev),
                         _int_table(lens, "lens", dev), max_len,
                         d ** -0.5 if scale is None else scale, lse.data_ptr(), 0, 0,
                         *_workspace(workspace, dev), _status_ptr(status, dev), before,
                         _int_table(prefix_lens, "prefix_lens", dev),
                         _int_table(groups, "groups", dev), prefix_table.shape[1], P, max_prefix,
                         max_group)
        st = _Fast.shared(a, _raw_stream(stream, dev))
        if st != KVX_OK:
            raise KvxError(st, "kvx_attend8_shared")
        return out, lse

    def _weights(self, w, R):
        """Pointer and row length of accumulated weights [R][heads][slots]."""
        shape = w.shape
        if w.dtype is not _Fast.f32 or w.device != self.device or len(shape) != 3 or \
                shape[0] != R or shape[1] != self.heads or not w.is_contiguous():
            raise ValueError(f"weights must be a contiguous fp32 [{R}][{self.heads}][slots] tensor "
                             f"on {self.device}")
        return w.data_ptr(), shape[2]

    def evict_workspace(self, *, num_requests, max_len, keep):
        """A workspace (uint8) for ``evict`` calls of at most these sizes that
        are ordered on one stream."""
        import torch
        a = Evict8Args()
        any_ptr = self.k_codes.data_ptr()                 # sizes only: never read
        a.cache = Cache8Desc(*self._head, 1, any_ptr)
        a.dst_table = a.lens = a.weights = a.kept = a.new_lens = any_ptr
        a.max_dst_blocks, a.weights_stride = 2 ** 31 - 1, max_len
        a.num_requests, a.max_len, a.keep = num_requests, max_len, keep
        need = kvx_evict8_workspace_bytes(a)
        if need == 0:
            raise KvxError(KVX_ERR_INVALID_ARG, "kvx_evict8_workspace_bytes")
        return torch.empty(need, dtype=torch.uint8, device=self.device)

    def evict(self, weights, block_table, lens, dst_table, *, max_len, keep, sinks=0, recent=0,
              kept=None, kept_weights=None, new_lens=None, workspace=None, status=None,
              stream=None):
        """Keep ``keep`` slots of each request and head: the first ``sinks``,
        the last ``recent`` and those of the largest ``weights``
        [R][heads][>= max_len]; move them into the blocks of ``dst_table`` (same
        pool, none of them read by this call).  Returns kept slots
        [R][heads][keep] (-1 beyond), their weights and the new lengths [R]."""
        dev = self.device
        _on_device(dev)
        table = self._table(block_table)
        R = block_table.shape[0]
        wptr, wstride = self._weights(weights, R)
        if lens.shape[0] != R or dst_table.dim() != 2 or dst_table.shape[0] != R:
            raise ValueError("lens, block_table and dst_table must hold the same requests")
        shape = (R, self.heads, keep)
        if kept is None:
            kept = _new(stream, shape, _Fast.i32, dev)
        elif tuple(kept.shape) != shape:
            raise ValueError("kept must be [R][heads][keep]")
        if kept_weights is None:
            kept_weights = _new(stream, shape, _Fast.f32, dev)
        elif kept_weights.dtype is not _Fast.f32 or kept_weights.device != dev or \
                tuple(kept_weights.shape) != shape or not kept_weights.is_contiguous():
            raise ValueError(f"kept_weights must be a contiguous fp32 [R][heads][keep] tensor on {dev}")
        if new_lens is None:
            new_lens = _new(stream, (R,), _Fast.i32, dev)
        elif new_lens.shape[0] != R:
            raise ValueError("new_lens must be [R]")
        if workspace is None:
            workspace = _on_stream(self.evict_workspace, stream, num_requests=R, max_len=max_len,
                                   keep=keep)
        a = _pack_evict(*table, _int_table(dst_table, "dst_table", dev, 2), dst_table.shape[1], R,
                        _int_table(lens, "lens", dev), max_len, keep, sinks, recent, wptr, wstride,
                        _int_table(kept, "kept", dev, 3), kept_weights.data_ptr(),
                        _int_table(new_lens, "new_lens", dev), *_workspace(workspace, dev),
                        _status_ptr(status, dev))
        st = _Fast.evict(a, _raw_stream(stream, dev))
        if st != KVX_OK:
            raise KvxError(st, "kvx_evict8")
        return kept, kept_weights, new_lens


def _cache_array(caches, num_blocks, device):
    """The caches as an array of ``kvx_cache8`` (kept by the caller for the call) and its address."""
    if not caches:
        return None, 0
    for c in caches:
        if c.num_blocks != num_blocks or c.device != device:
            raise ValueError(f"caches must hold {num_blocks} blocks on {device}")
    raw = ctypes.c_char_p(b"".join([c._packed for c in caches]))
    return raw, ctypes.cast(raw, ctypes.c_void_p).value


class Pages:
    """References to the pages (blocks) of a pool: ``refs`` [num_blocks] int32
    counts the entries of block tables that hold each, 0 for a free page.  A
    table's entries of -1 hold none.  The caches of all layers share one set of
    tables and one ``Pages``.  ``Pages.empty`` starts with all pages free."""

    def __init__(self, refs, block_size):
        import torch
        if refs.dtype != torch.int32 or refs.dim() != 1 or not refs.is_contiguous():
            raise ValueError("refs must be a contiguous 1-D int32 tensor")
        self.refs, self.block_size, self.device = refs, int(block_size), refs.device
        self.num_blocks = refs.shape[0]
        self._index = refs.device.index

    @classmethod
    def empty(cls, num_blocks, block_size, device="cuda"):
        import torch
        return cls(torch.zeros(num_blocks, dtype=torch.int32, device=device), block_size)

    def workspace(self):
        """A workspace (uint8) for ``reserve`` and ``compact`` calls that are
        ordered on one stream."""
        import torch
        need = kvx_pages_workspace_bytes(self.num_blocks)
        if need == 0:
            raise KvxError(KVX_ERR_INVALID_ARG, "kvx_pages_workspace_bytes")
        return torch.empty(need, dtype=torch.uint8, device=self.device)

    def _ready(self):
        """The pool's device, which has to be the current one."""
        if _Fast.torch is None or _Fast.device() != self._index:
            _on_device(self.device)
        return self.device

    def _rows(self, table, lens):
        """Rows, width and pointer of a table, and the pointer of the rows' lengths."""
        ptr = _int_table(table, "table", self.device, 2)
        R, width = table.shape
        if lens.shape[0] != R:
            raise ValueError("lens and table must hold the same rows")
        return R, width, ptr, _int_table(lens, "lens", self.device)

    def fork(self, table, lens, parents, *, new_table=None, new_lens=None, status=None, stream=None):
        """New rows in place of those of ``table`` [R][width]: row n continues
        row parents[n] (-1: an empty row) and shares the pages that its length
        covers.  The old rows hold nothing afterwards.  Returns (new_table
        [N][width], new_lens [N]), which overlap nothing that is read."""
        dev = self._ready()
        R, width, ptr, len_ptr = self._rows(table, lens)
        parent = _int_table(parents, "parents", dev)
        N = parents.shape[0]
        if new_table is None:
            new_table = _new(stream, (N, width), _Fast.i32, dev)
            to = new_table.data_ptr()
        else:
            to = _int_table(new_table, "new_table", dev, 2)
            if tuple(new_table.shape) != (N, width):
                raise ValueError("new_table must be [N][width]")
        if new_lens is None:
            new_lens = _new(stream, (N,), _Fast.i32, dev)
            to_lens = new_lens.data_ptr()
        else:
            to_lens = _int_table(new_lens, "new_lens", dev)
            if new_lens.shape[0] != N:
                raise ValueError("new_lens must be [N]")
        a = _pack_fork(self.refs.data_ptr(), self.num_blocks, self.block_size, R, width, ptr,
                       len_ptr, parent, N, to, to_lens, _status_ptr(status, dev))
        st = _Fast.fork(a, _raw_stream(stream, dev))
        if st != KVX_OK:
            raise KvxError(st, "kvx_pages_fork")
        return new_table, new_lens

    def free(self, table, *, status=None, stream=None):
        """The rows of ``table`` (some rows of one: a slice) release their pages;
        their entries become -1."""
        dev = self._ready()
        ptr = _int_table(table, "table", dev, 2)
        a = PagesFreeArgs(self.refs.data_ptr(), self.num_blocks, *table.shape, ptr,
                          _status_ptr(status, dev))
        st = kvx_pages_free(a, _raw_stream(stream, dev))
        if st != KVX_OK:
            raise KvxError(st, "kvx_pages_free")

    def reserve(self, table, lens, new=1, *, max_new=None, caches=(), copies=None, workspace=None,
                status=None, stream=None):
        """Make slots lens .. lens + new - 1 of every row of ``table`` writable:
        each behind a page of the row's own, taken from the free ones where
        there is none or others hold it too; a page that holds slots of the
        row is then copied in all ``caches``.  ``new`` is one number, or
        one for each row (int32 tensor, at most ``max_new``).  ``copies`` [R][2]
        (int32) receives the copied pages, from and to (-1: none).  With too few
        free pages none is taken or copied, and ``status`` tells
        (KVX_FLAG_NO_PAGES): then only entries that are no pages change, to -1."""
        dev = self._ready()
        R, width, ptr, len_ptr = self._rows(table, lens)
        add = 0
        if isinstance(new, int):
            most = new
        else:
            add = _int_table(new, "new", dev)
            if new.shape[0] != R:
                raise ValueError("new must hold one entry for each row")
            most = width * self.block_size if max_new is None else max_new
        copy_ptr = _int_table(copies, "copies", dev, 2)
        if copy_ptr and tuple(copies.shape) != (R, 2):
            raise ValueError("copies must be [R][2]")
        if workspace is None:
            workspace = _on_stream(self.workspace, stream)
        keep, array = _cache_array(caches, self.num_blocks, dev)
        a = _pack_reserve(self.refs.data_ptr(), self.num_blocks, self.block_size, R, width, ptr,
                          len_ptr, add, most, copy_ptr, array, len(caches),
                          *_workspace(workspace, dev), _status_ptr(status, dev))
        st = _Fast.reserve(a, _raw_stream(stream, dev))
        if st != KVX_OK:
            raise KvxError(st, "kvx_pages_reserve")

    def compact(self, tables, caches=(), *, used=None, moved=None, workspace=None, status=None,
                stream=None):
        """Move the held pages to the lowest numbers, in all ``caches``, and
        rewrite ``tables`` (up to eight int32 tensors, which hold all
        references and do not overlap).  Returns (used [1], moved [num_blocks]): how many pages are
        held, and each page's new number (-1: it is free)."""
        dev = self._ready()
        if used is None:
            used = _new(stream, (1,), _Fast.i32, dev)
            used_ptr = used.data_ptr()
        else:
            used_ptr = _int_table(used, "used", dev)
        if moved is None:
            moved = _new(stream, (self.num_blocks,), _Fast.i32, dev)
            moved_ptr = moved.data_ptr()
        else:
            moved_ptr = _int_table(moved, "moved", dev)
            if moved.shape[0] != self.num_blocks:
                raise ValueError("moved must be [num_blocks]")
        if workspace is None:
            workspace = _on_stream(self.workspace, stream)
        keep, array = _cache_array(caches, self.num_blocks, dev)
        n = len(tables)
        lists = (ctypes.c_int64 * (2 * n + 1))(
            *[_int_table(t, "tables", dev, t.dim()) for t in tables], *[t.numel() for t in tables])
        at = ctypes.addressof(lists)
        a = _pack_compact(self.refs.data_ptr(), self.num_blocks, self.block_size, at, at + 8 * n, n,
                          used_ptr, moved_ptr, array, len(caches), *_workspace(workspace, dev), _status_ptr(status, dev))
        st = _Fast.compact(a, _raw_stream(stream, dev))
        if st != KVX_OK:
            raise KvxError(st, "kvx_pages_compact")
        return used, moved


def copy_pages(caches, pairs, count=None, *, status=None, stream=None):
    """Copy whole pages, codes and scales, in all ``caches`` (``kvx_cache8_copy``):
    from page pairs[i][0] to page pairs[i][1] (pairs with a negative one are
    skipped); with ``count`` [1] only the first count[0]."""
    if not caches:
        return
    dev = caches[0].device
    _on_device(dev)
    keep, array = _cache_array(caches, caches[0].num_blocks, dev)
    ptr = _int_table(pairs, "pairs", dev, 2)
    if pairs.shape[1] != 2:
        raise ValueError("pairs must be [pairs][2]")
    a = Cache8CopyArgs(array, len(caches), ptr, pairs.shape[0], _int_table(count, "count", dev),
                       _status_ptr(status, dev))
    st = kvx_cache8_copy(a, _raw_stream(stream, dev))
    if st != KVX_OK:
        raise KvxError(st, "kvx_cache8_copy")


def beam_workspace(*, requests, beams, vocab, out=None, device="cuda"):
    """A workspace (uint8) for ``beam_select`` calls of at most these sizes that
    are ordered on one stream."""
    import torch
    a = BeamArgs(dtype=KVX_F32, num_requests=requests, beams=beams,
                 out_beams=beams if out is None else out, vocab=vocab, eos=-1)
    need = kvx_beam_workspace_bytes(a)
    if need == 0:
        raise KvxError(KVX_ERR_INVALID_ARG, "kvx_beam_workspace_bytes")
    return torch.empty(need, dtype=torch.uint8, device=device)


def beam_select(logits, scores, *, beams=None, eos=None, done=None, tokens=None, parents=None,
                new_scores=None, new_done=None, workspace=None, status=None, stream=None):
    """Beam search's selection (``kvx_beam_select``): of the candidates of each
    request, scores[b][k] + log_softmax(logits[b * K + k])[v], the ``beams`` (K) of
    the largest score: within a beam by logit, equal ones by v; equal scores of
    different beams by k.  ``logits`` [B * K][V] (fp32 or bf16, unit stride inside a row), ``scores`` [B][K] fp32 (-inf: no beam); beams that
    are ``done`` [B][K] (bool) have one candidate, ``eos`` with the score they
    have.  Returns (tokens, parents, scores, done) [B][beams]: parents are rows of
    logits, as ``Pages.fork`` takes them (-1, with a score of -inf: no candidate);
    done is None without ``eos``."""
    dev = logits.device
    _on_device(dev)
    if logits.dim() != 2 or logits.stride(1) != 1 and logits.shape[1] > 1:
        raise ValueError("logits must be [beams][vocab] with unit stride inside a row")
    if scores.dtype is not _Fast.f32 or scores.dim() != 2 or scores.device != dev or \
            not scores.is_contiguous() or scores.numel() != logits.shape[0]:
        raise ValueError(f"scores must be a contiguous fp32 [requests][beams] tensor on {dev}, "
                         f"one for each row of logits")
    B, K = scores.shape
    N = K if beams is None else beams
    torch = _Fast.torch
    done_ptr = new_done_ptr = 0
    if done is not None:
        if eos is None:
            raise ValueError("done needs eos")
        done_ptr = _flags(done, "done", (B, K), dev)
    tokens = _output(tokens, "tokens", (B, N), _Fast.i32, dev, stream)
    parents = _output(parents, "parents", (B, N), _Fast.i32, dev, stream)
    new_scores = _output(new_scores, "new_scores", (B, N), _Fast.f32, dev, stream)
    if eos is not None:
        if new_done is None:
            new_done = _new(stream, (B, N), torch.bool, dev)
        new_done_ptr = _flags(new_done, "new_done", (B, N), dev)
    elif new_done is not None:
        raise ValueError("new_done needs eos")
    if workspace is None:
        workspace = _on_stream(beam_workspace, stream, requests=B, beams=K, vocab=logits.shape[1],
                               out=N, device=dev)
    a = _pack_beam(logits.data_ptr(), logits.stride(0), _code_of(logits.dtype), B, K, N,
                   logits.shape[1], -1 if eos is None else eos, scores.data_ptr(), done_ptr,
                   tokens.data_ptr(), parents.data_ptr(), new_scores.data_ptr(), new_done_ptr,
                   *_workspace(workspace, dev), _status_ptr(status, dev))
    st = _Fast.beam(a, _raw_stream(stream, dev))
    if st != KVX_OK:
        raise KvxError(st, "kvx_beam_select")
    return tokens, parents, new_scores, new_done


def _flags(t, name, shape, device):
    """Data pointer of a contiguous bool (or uint8) tensor."""
    torch = _Fast.torch
    if t.dtype not in (torch.bool, torch.uint8) or tuple(t.shape) != shape or t.device != device or \
            not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bool {list(shape)} tensor on {device}")
    return t.data_ptr()


def _output(t, name, shape, dtype, device, stream):
    """An output, checked or allocated."""
    if t is None:
        return _new(stream, shape, dtype, device)
    if t.dtype is not dtype or tuple(t.shape) != shape or t.device != device or \
            not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on {device}")
    return t


def _new(stream, shape, dtype, device):
    """An uninitialised tensor for a call on ``stream``."""
    if stream is None:
        return _Fast.empty(shape, dtype=dtype, device=device)
    return _on_stream(_Fast.empty, stream, shape, dtype=dtype, device=device)


def _on_stream(make, stream, *args, **kw):
    """``make(...)`` with ``stream`` current: a tensor allocated for a call on
    another stream must come from that stream's memory, or it could be handed
    out again before the call is done."""
    import torch
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        return make(*args, **kw)
