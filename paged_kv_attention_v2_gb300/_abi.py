"""ctypes view of include/pa_decode.h and include/pa_cache.h, and loading of libpa_decode.so.

Loading fails loudly when the library has not been built: there is no other
implementation behind this package.
"""
from __future__ import annotations

import ctypes
import struct
from pathlib import Path

PKG = Path(__file__).resolve().parent
LIB_PATH = PKG / "_build" / "libpa_decode.so"

PA_OK = 0
PA_ERR_INVALID_ARG = 1
PA_ERR_UNSUPPORTED = 2
PA_ERR_WORKSPACE = 3
PA_ERR_LAUNCH = 4
PA_ERR_DEVICE_CHECK = 5
PA_ERR_DEVICE_TIMEOUT = 6

PA_DTYPE_F32, PA_DTYPE_F16, PA_DTYPE_BF16 = 0, 1, 2
PA_LAYOUT_SPLIT, PA_LAYOUT_NHD = 0, 1
PA_MODE_AUTO, PA_MODE_V1, PA_MODE_V2 = 0, 1, 2
PA_KV_SAME, PA_KV_FP8_E4M3, PA_KV_FP8_E5M2, PA_KV_FP4_E2M1 = 0, 3, 4, 5

PA_DEVERR_BLOCK_ID = 1
PA_DEVERR_SEQ_LEN = 2
PA_DEVERR_TIMEOUT = 4
PA_DEVERR_QUERY_RANGE = 8
PA_DEVERR_POOL = 16
PA_DEVERR_SLOT = 32

PA_PARTITION_SIZE = 512
PA_BLOCK_SIZE = 16

# every function include/pa_decode.h and include/pa_cache.h declare
EXPORTED = ("pa_decode", "pa_max_num_partitions", "pa_workspace_elems", "pa_choose_mode",
            "pa_choose_mode_for_lengths", "pa_workspace_bytes", "pa_partition_size", "pa_plan",
            "pa_status_str", "pa_version", "pa_decode_static_workspace", "pa_debug_withhold_page",
            "pa_build_tables", "pa_append_kv", "pa_diff_decode", "pa_diff_plan",
            "pa_add_weights", "pa_select_tokens", "pa_compact_kv")

PA_STATIC_WORKSPACE_FLOATS = 4 * 1024 * 1024
PA_FUSED_MAX_PARTITIONS = 8


class PaDecodeArgs(ctypes.Structure):
    _fields_ = [
        ("out", ctypes.c_void_p),
        ("query", ctypes.c_void_p),
        ("key_cache", ctypes.c_void_p),
        ("value_cache", ctypes.c_void_p),
        ("block_tables", ctypes.c_void_p),
        ("seq_lens", ctypes.c_void_p),
        ("num_seqs", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_size", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("max_seq_len", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("softcap", ctypes.c_float),
        ("alibi_slopes", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
        ("layout", ctypes.c_int32),
        ("mode", ctypes.c_int32),
        ("exp_sums", ctypes.c_void_p),
        ("max_logits", ctypes.c_void_p),
        ("tmp_out", ctypes.c_void_p),
        ("dev_error", ctypes.c_void_p),
        ("event_main_begin", ctypes.c_void_p),
        ("event_main_end", ctypes.c_void_p),
        ("partition_counters", ctypes.c_void_p),
        ("sliding_window", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
        ("query_start", ctypes.c_void_p),
        ("num_query_tokens", ctypes.c_int32),
        ("max_query_len", ctypes.c_int32),
        ("seq_lens_host", ctypes.c_void_p),
        ("tile_counters", ctypes.c_void_p),
        ("metadata_ready", ctypes.c_int32),
        ("relative_max", ctypes.c_int32),
    ]


class PaLaunchPlan(ctypes.Structure):
    _fields_ = [
        ("mode", ctypes.c_int32),
        ("merge_in_kernel", ctypes.c_int32),
        ("kernels", ctypes.c_int32),
        ("ctas_per_sm", ctypes.c_int32),
        ("grid", ctypes.c_int32),
        ("dynamic_schedule", ctypes.c_int32),
        ("partition_tokens", ctypes.c_int32),
        ("tiles", ctypes.c_int64),
    ]


class PaDiffArgs(ctypes.Structure):
    _fields_ = [
        ("decode", PaDecodeArgs),
        ("lambdas", ctypes.c_void_p),
        ("lambda_row_stride", ctypes.c_int64),
        ("norm_weight", ctypes.c_void_p),
        ("norm_eps", ctypes.c_float),
        ("out_scale", ctypes.c_float),
        ("norm", ctypes.c_int32),
    ]


class PaTablesArgs(ctypes.Structure):
    _fields_ = [
        ("block_tables", ctypes.c_void_p),
        ("seq_lens", ctypes.c_void_p),
        ("keep_lens", ctypes.c_void_p),
        ("query_start", ctypes.c_void_p),
        ("free_ring", ctypes.c_void_p),
        ("pool_state", ctypes.c_void_p),
        ("slots", ctypes.c_void_p),
        ("positions", ctypes.c_void_p),
        ("new_seq_lens", ctypes.c_void_p),
        ("new_pool_state", ctypes.c_void_p),
        ("num_seqs", ctypes.c_int32),
        ("num_tokens", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("max_seq_len", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("dev_error", ctypes.c_void_p),
        ("done_counter", ctypes.c_void_p),
    ]


class PaAppendArgs(ctypes.Structure):
    _fields_ = [
        ("key", ctypes.c_void_p),
        ("value", ctypes.c_void_p),
        ("key_cache", ctypes.c_void_p),
        ("value_cache", ctypes.c_void_p),
        ("slots", ctypes.c_void_p),
        ("key_stride", ctypes.c_int64),
        ("key_head_stride", ctypes.c_int64),
        ("value_stride", ctypes.c_int64),
        ("value_head_stride", ctypes.c_int64),
        ("num_tokens", ctypes.c_int32),
        ("num_key_heads", ctypes.c_int32),
        ("key_head_size", ctypes.c_int32),
        ("num_value_heads", ctypes.c_int32),
        ("value_head_size", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("layout", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
        ("dev_error", ctypes.c_void_p),
    ]


class PaWeightsArgs(ctypes.Structure):
    _fields_ = [
        ("scores", ctypes.c_void_p),
        ("query", ctypes.c_void_p),
        ("key_cache", ctypes.c_void_p),
        ("block_tables", ctypes.c_void_p),
        ("seq_lens", ctypes.c_void_p),
        ("exp_sums", ctypes.c_void_p),
        ("max_logits", ctypes.c_void_p),
        ("alibi_slopes", ctypes.c_void_p),
        ("query_start", ctypes.c_void_p),
        ("dev_error", ctypes.c_void_p),
        ("num_seqs", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_size", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("max_seq_len", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("num_query_tokens", ctypes.c_int32),
        ("max_query_len", ctypes.c_int32),
        ("sliding_window", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("layout", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("softcap", ctypes.c_float),
        ("k_scale", ctypes.c_float),
        ("decay", ctypes.c_float),
        ("relative_max", ctypes.c_int32),
    ]


class PaSelectArgs(ctypes.Structure):
    _fields_ = [
        ("kept", ctypes.c_void_p),
        ("new_seq_lens", ctypes.c_void_p),
        ("scores", ctypes.c_void_p),
        ("block_tables", ctypes.c_void_p),
        ("seq_lens", ctypes.c_void_p),
        ("budgets", ctypes.c_void_p),
        ("dev_error", ctypes.c_void_p),
        ("num_seqs", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("max_seq_len", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("max_budget", ctypes.c_int32),
        ("sink", ctypes.c_int32),
        ("recent", ctypes.c_int32),
    ]


class PaCompactArgs(ctypes.Structure):
    _fields_ = [
        ("key_cache", ctypes.c_void_p),
        ("value_cache", ctypes.c_void_p),
        ("scores", ctypes.c_void_p),
        ("block_tables", ctypes.c_void_p),
        ("kept", ctypes.c_void_p),
        ("new_seq_lens", ctypes.c_void_p),
        ("dev_error", ctypes.c_void_p),
        ("num_seqs", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("max_budget", ctypes.c_int32),
        ("num_key_heads", ctypes.c_int32),
        ("key_head_size", ctypes.c_int32),
        ("num_value_heads", ctypes.c_int32),
        ("value_head_size", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("layout", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
    ]


def sliding_window(window_left: int) -> int:
    """The structs' sliding_window of a window_left: 0 (off) for negative ones, and for ones
    that reach over any length."""
    return int(window_left) + 1 if 0 <= window_left < 2 ** 31 - 1 else 0


_CODES = {ctypes.c_void_p: "P", ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_float: "f"}


def packer(cls) -> struct.Struct:
    """struct.Struct with the layout of an argument struct (nested ones field by
    field), the same as the C compiler's: packing the fields' values into bytes
    takes a fraction of the time that filling a ctypes structure does."""
    def codes(c):
        for _, t in c._fields_:
            yield from codes(t) if issubclass(t, ctypes.Structure) else _CODES[t]
    return struct.Struct("@" + "".join(codes(cls)) + "0P")  # padded at the end like the struct


_lib = None


class LibraryMissing(RuntimeError):
    pass


def load(path: Path | None = None):
    """Load libpa_decode.so (built by paged_kv_attention_v2_gb300.build)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = Path(path) if path else LIB_PATH
    if not p.exists():
        raise LibraryMissing(
            f"{p} is missing: build it with `python -m paged_kv_attention_v2_gb300.build` "
            "(or __graft_entry__.build()); there is no fallback implementation")
    lib = ctypes.CDLL(str(p))
    # argument structs come as structures (byref) or as packed bytes
    lib.pa_decode.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib.pa_decode.restype = ctypes.c_int
    lib.pa_max_num_partitions.argtypes = [ctypes.c_int32]
    lib.pa_max_num_partitions.restype = ctypes.c_int32
    lib.pa_workspace_elems.argtypes = [ctypes.c_int32] * 4 + [ctypes.POINTER(ctypes.c_int64)] * 2
    lib.pa_workspace_elems.restype = ctypes.c_int
    lib.pa_choose_mode.argtypes = [ctypes.c_int32] * 5
    lib.pa_choose_mode.restype = ctypes.c_int32
    lib.pa_workspace_bytes.argtypes = [ctypes.c_int32] * 4
    lib.pa_workspace_bytes.restype = ctypes.c_size_t
    lib.pa_partition_size.argtypes = []
    lib.pa_partition_size.restype = ctypes.c_int32
    lib.pa_choose_mode_for_lengths.argtypes = [ctypes.c_int32] * 5 + [ctypes.c_void_p]
    lib.pa_choose_mode_for_lengths.restype = ctypes.c_int32
    lib.pa_status_str.argtypes = [ctypes.c_int32]
    lib.pa_status_str.restype = ctypes.c_char_p
    lib.pa_version.restype = ctypes.c_int32
    lib.pa_decode_static_workspace.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib.pa_decode_static_workspace.restype = ctypes.c_int
    lib.pa_plan.argtypes = [ctypes.POINTER(PaDecodeArgs), ctypes.POINTER(PaLaunchPlan)]
    lib.pa_plan.restype = ctypes.c_int
    lib.pa_debug_withhold_page.argtypes = [ctypes.c_int32, ctypes.c_int64]
    lib.pa_debug_withhold_page.restype = ctypes.c_int
    lib.pa_diff_decode.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib.pa_diff_decode.restype = ctypes.c_int
    lib.pa_diff_plan.argtypes = [ctypes.POINTER(PaDiffArgs), ctypes.POINTER(PaLaunchPlan)]
    lib.pa_diff_plan.restype = ctypes.c_int
    lib.pa_build_tables.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib.pa_build_tables.restype = ctypes.c_int
    lib.pa_append_kv.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib.pa_append_kv.restype = ctypes.c_int
    for fn in (lib.pa_add_weights, lib.pa_select_tokens, lib.pa_compact_kv):
        fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
        fn.restype = ctypes.c_int
    if path is None:
        _lib = lib
    return lib
