"""ctypes declarations of the libspecverify C ABI (include/specverify.h).

Loading fails loudly when the shared library is missing: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecverify.so")

c_int, c_i32p, c_i64, c_f32, c_f64 = ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_double
c_vp, c_size = ctypes.c_void_p, ctypes.c_size_t

SV_OK, SV_ERR_INVALID_ARG, SV_ERR_CUDA, SV_ERR_NONFINITE, SV_ERR_TIMEOUT, SV_ERR_WORKSPACE, SV_ERR_BAD_TOKEN, SV_ERR_NO_PAGE = range(8)
SV_F32, SV_BF16 = 0, 1
SV_DEBUG_FIELDS = 8
SV_MAX_K = 32
SV_STATIC_SCRATCH_BYTES = 32 << 20
SV_ACCEPT_DIVERGENCE, SV_ACCEPT_ASSISTED = 0, 1   # sv_accept_mode   # scratch array behind sv_verify_static
SV_MAX_TREE = 128
SV_KV_MAX_HEAD_DIM = 256
SV_ROPE_STYLES = {"half": 0, "interleaved": 1}   # sv_rope_style
SV_ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "turns": 3, "dims": 4}   # sv_rope_scaling
DBG = dict(lse_q=0, lse_p=1, q_s=2, p_s=3, ratio=4, mass_q=5, mass_p=6, R=7)


class SvStats(ctypes.Structure):
    _fields_ = [("status", ctypes.c_int32), ("error_index", ctypes.c_int32), ("rows", ctypes.c_int64),
                ("accept_tests", ctypes.c_int64), ("draws", ctypes.c_int64), ("reresolved", ctypes.c_int64),
                ("near_boundary", ctypes.c_int64), ("unresolved", ctypes.c_int64)]


class SvKvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("slot_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class SvKvBatch(ctypes.Structure):
    _fields_ = [("context_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("row_start", ctypes.c_void_p),
                ("parents", ctypes.c_void_p), ("table_pitch", ctypes.c_int64), ("max_pages", ctypes.c_int32),
                ("B", ctypes.c_int32), ("n", ctypes.c_int32), ("rows", ctypes.c_int32)]


class SvKvCache8(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("scale_page_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class SvKvPool(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("layer_stride", ctypes.c_int64), ("page_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("head_bytes", ctypes.c_int64), ("scale_layer_stride", ctypes.c_int64),
                ("scale_page_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64), ("n_layers", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32)]


STATS_FIELDS = [f for f, _ in SvStats._fields_]
STATS_BYTES = ctypes.sizeof(SvStats)

c_kv, c_bt = ctypes.POINTER(SvKvCache), ctypes.POINTER(SvKvBatch)
c_kv8, c_pool = ctypes.POINTER(SvKvCache8), ctypes.POINTER(SvKvPool)

# name -> (restype, argtypes); the order follows the header.
SIGNATURES = {
    "sv_status_string": (ctypes.c_char_p, [c_int]),
    "sv_version": (c_int, []),
    "sv_verify_workspace_size": (c_size, [c_int, c_int, c_int]),
    "sv_verify": (c_int, [c_vp, c_i64, c_vp, c_i64, c_int, c_int, c_vp, c_vp, c_int, c_int, c_int, c_vp, c_vp,
                          c_vp, c_int, c_f32, c_vp, c_vp, c_vp, c_vp, c_vp, c_size, c_vp]),
    "sv_verify_host_workspace_size": (c_size, [c_int, c_int, c_int, c_int]),
    "sv_verify_host": (c_int, [c_vp, c_i64, c_vp, c_i64, c_int, c_int, c_vp, c_vp, c_int, c_int, c_int, c_vp, c_vp,
                               c_vp, c_int, c_f32, c_vp, c_vp, c_vp, c_vp, c_size, c_vp, c_vp]),
    "sv_verify_lazy": (c_int, [c_vp, c_i64, c_vp, c_i64, c_int, c_int, c_vp, c_vp, c_int, c_int, c_int, c_vp, c_vp,
                               c_vp, c_int, c_f32, c_vp, c_vp, c_vp, c_vp, c_vp, c_size, c_vp]),
    "sv_verify_static": (c_int, [c_vp, c_i64, c_vp, c_i64, c_int, c_int, c_vp, c_vp, c_int, c_int, c_int, c_vp,
                                 c_vp, c_vp, c_int, c_f32, c_vp, c_vp, c_vp, c_vp, c_vp]),
    "sv_tree_verify_workspace_size": (c_size, [c_int, c_int, c_int]),
    "sv_tree_verify": (c_int, [c_vp, c_i64, c_vp, c_i64, c_int, c_vp, c_vp, c_vp, c_int, c_int, c_int, c_vp, c_vp, c_vp,
                               c_vp, c_vp, c_vp, c_size, c_vp]),
    "sv_tree_reuse": (c_int, [c_vp, c_vp, c_int, c_vp, c_vp, c_int, c_int, c_vp, c_vp]),
    "sv_fuzzy_verify_workspace_size": (c_size, [c_int, c_int, c_int]),
    "sv_fuzzy_verify": (c_int, [c_vp, c_i64, c_vp, c_i64, c_int, c_int, c_vp, c_vp, c_int, c_int, c_int, c_vp, c_f32,
                                c_int, c_vp, c_vp, c_vp, c_vp, c_vp, c_size, c_vp]),
    "sv_saguaro_sample_workspace_size": (c_size, [c_int, c_int, c_int]),
    "sv_saguaro_sample": (c_int, [c_vp, c_i64, c_int, c_int, c_int, c_int, c_int, c_vp, c_vp, c_vp, c_int, c_f32,
                                  c_vp, c_vp, c_vp, c_vp, c_vp, c_size, c_vp]),
    "sv_fanout": (c_int, [c_f64, c_f64, c_f64, c_int, c_vp, c_vp]),
    "sv_cache_keys_workspace_size": (c_size, [c_int, c_int, c_int]),
    "sv_cache_keys": (c_int, [c_vp, c_i64, c_int, c_int, c_vp, c_vp, c_int, c_int, c_int, c_vp, c_vp, c_vp, c_size,
                              c_vp]),
    "sv_cache_lookup": (c_int, [c_vp, c_vp, c_vp, c_vp, c_int, c_int, c_vp, c_vp]),
    "sv_topk_rows_workspace_size": (c_size, [c_int, c_int]),
    "sv_topk_rows": (c_int, [c_vp, c_i64, c_int, c_int, c_int, c_int, c_vp, c_vp, c_vp, c_vp, c_vp, c_size, c_vp]),
    "sv_mirror_reuse": (c_int, [c_vp, c_vp, c_vp, c_int, c_int, c_int, c_vp, c_vp]),
    "sv_rope_frequencies": (c_int, [c_int, c_f64, c_int, c_f64, c_f64, c_f64, c_i64, c_vp, c_vp]),
    "sv_rope": (c_int, [c_vp, c_i64, c_i64, c_vp, c_i64, c_i64, c_int, c_i64, c_int, c_int, c_vp, c_vp, c_int, c_int,
                        c_f32, c_int, c_vp]),
    "sv_kv_append": (c_int, [c_kv, c_bt, c_vp, c_i64, c_i64, c_vp, c_i64, c_i64, c_int, c_vp, c_i64, c_i64, c_vp,
                             c_i64, c_i64, c_vp, c_int, c_int, c_f32, c_vp, c_vp]),
    "sv_kv_attend_workspace_size": (c_size, [c_i64, c_int, c_int, c_int, c_int]),
    "sv_kv_attend": (c_int, [c_kv, c_bt, c_vp, c_i64, c_i64, c_int, c_f32, c_vp, c_vp, c_int, c_vp, c_i64, c_i64, c_vp,
                             c_vp, c_vp, c_size, c_vp]),
    "sv_kv_commit": (c_int, [c_kv, c_bt, c_int, c_i64, c_vp, c_vp, c_vp, c_vp, c_vp]),
    "sv_kv_append8": (c_int, [c_kv8, c_bt, c_int, c_vp, c_i64, c_i64, c_vp, c_i64, c_i64, c_int, c_vp, c_i64, c_i64, c_vp,
                              c_i64, c_i64, c_vp, c_int, c_int, c_f32, c_vp, c_vp]),
    "sv_kv_attend8": (c_int, [c_kv8, c_bt, c_int, c_vp, c_i64, c_i64, c_int, c_f32, c_vp, c_vp, c_int, c_vp, c_i64, c_i64,
                              c_vp, c_vp, c_vp, c_size, c_vp]),
    "sv_kv_commit8": (c_int, [c_kv8, c_bt, c_int, c_i64, c_i64, c_vp, c_vp, c_vp, c_vp, c_vp]),
    "sv_kv_fork_workspace_size": (c_size, [c_int, c_int]),
    "sv_kv_fork": (c_int, [c_pool, c_vp, c_vp, c_vp, c_i64, c_int, c_int, c_vp, c_int, c_int, c_vp, c_vp, c_i64, c_vp, c_vp,
                           c_vp, c_size, c_vp]),
    "sv_kv_compact_workspace_size": (c_size, [c_int]),
    "sv_kv_compact": (c_int, [c_pool, c_vp, c_vp, c_i64, c_int, c_int, c_vp, c_vp, c_i64, c_vp, c_vp, c_vp, c_vp, c_size,
                              c_vp]),
    "sv_stream_capture_id": (ctypes.c_uint64, [c_vp]),
    "sv_set_profile_events": (None, [c_vp, c_vp]),
    "sv_selftest_timeout": (c_int, [c_i64, c_vp, c_vp]),
    "sv_selftest_attend_stall": (None, [c_i64]),
    "sv_selftest_exp2": (c_int, [c_f64, c_f64, c_i64, c_vp, c_vp]),
    "sv_selftest_exp2_all": (c_int, [c_f32, c_f32, c_vp, c_vp]),
}

# The structures as bytes, in the layout of SvKvCache, SvKvCache8, SvKvPool and SvKvBatch: packing one takes a fifth of the time of
# filling a ctypes structure.
KV_CACHE = struct.Struct("PPqqqiiiii4x")
KV_CACHE8 = struct.Struct("PPPPqqqqqiiii")
KV_POOL = struct.Struct("PPPPqqqqqqqqiiii")
KV_BATCH = struct.Struct("PPPPqiiii")
_packed = None


def load_packed():
    """The library with the structures of the cache's calls passed as bytes (KV_CACHE, KV_CACHE8, KV_POOL, KV_BATCH)."""
    global _packed
    if _packed is None:
        load()
        lib = ctypes.CDLL(LIB_PATH)
        for name in ("sv_kv_append", "sv_kv_attend", "sv_kv_commit", "sv_kv_append8", "sv_kv_attend8", "sv_kv_commit8", "sv_kv_fork",
                     "sv_kv_compact"):
            res, args = SIGNATURES[name]
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = [ctypes.c_char_p if a in (c_kv, c_kv8, c_pool, c_bt) else a for a in args]
        _packed = lib
    return _packed


_lib = None


def load(path: str = LIB_PATH):
    """Load libspecverify and declare every entry point; raise if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libspecverify is not built ({path} missing); run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load().sv_status_string(code).decode()


class SvError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {status_string(code)} ({code})")
        self.code = code


def check(fn: str, code: int):
    if code != SV_OK:
        raise SvError(fn, code)
