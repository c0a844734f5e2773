"""Differential attention over the paged cache: Python binding of pa_diff_decode.

    ws = alloc_diff_workspace(rows, num_heads, head_size, max_seq_len, query.device)
    pa_diff_decode(out, query, key_cache, value_cache, block_tables, seq_lens, lambdas=lam,
                   num_kv_heads=..., scale=..., max_seq_len=..., norm_weight=w, out_scale=1 - lambda_init, **ws)
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import _abi
from .cache import _CACHE, _DTYPE, _KV, _LAYOUT, _PAGE, _call, _ints, _pointer

_DIFF = _abi.packer(_abi.PaDiffArgs)
_MODE = {"auto": _abi.PA_MODE_AUTO, "v1": _abi.PA_MODE_V1, "v2": _abi.PA_MODE_V2}


def alloc_diff_workspace(rows: int, num_heads: int, head_size: int, max_seq_len: int, device,
                         num_seqs: int | None = None, num_kv_heads: int | None = None,
                         tile_counters: bool = False) -> dict:
    """torch-allocated v2 workspace of pa_diff_decode for `rows` query rows:
    exp_sums and max_logits [rows, num_heads, 2, P], tmp_out [rows, num_heads, 2,
    P, 2 * head_size]; zeroed partition_counters when num_seqs and num_kv_heads
    are given (merge inside the partition kernel) and zeroed tile_counters when
    asked for (dynamic tile schedule)."""
    parts = int(_abi.load().pa_max_num_partitions(int(max_seq_len)))
    real = lambda *s: torch.empty(s, dtype=torch.float32, device=device)  # noqa: E731
    ws = {"exp_sums": real(rows, num_heads, 2, parts), "max_logits": real(rows, num_heads, 2, parts),
          "tmp_out": real(rows, num_heads, 2, parts, 2 * head_size)}
    if num_seqs is not None and num_kv_heads is not None:
        ws["partition_counters"] = torch.zeros((num_seqs, num_kv_heads), dtype=torch.int32, device=device)
    if tile_counters:
        ws["tile_counters"] = torch.zeros(2, dtype=torch.int32, device=device)
    return ws


def _floats(name: str, t, device: int, numel: int = -1, room: bool = False) -> int:
    return _pointer(name, t, torch.float32, device, numel, room)


def _pack_diff(out, query, key_cache, value_cache, block_tables, seq_lens, lambdas, num_kv_heads, scale, max_seq_len,
               norm=True, norm_weight=None, norm_eps=1e-5, out_scale=1.0, alibi_slopes=None, softcap=0.0,
               layout="split", mode="auto", exp_sums=None, max_logits=None, tmp_out=None, dev_error=None,
               event_begin=None, event_end=None, partition_counters=None, window_left=-1, kv_dtype=None, k_scale=1.0,
               v_scale=1.0, query_start=None, max_query_len=None, seq_lens_host=None, tile_counters=None,
               metadata_ready=False):
    """The packed arguments, and what has to live until the call has been made."""
    device, dtype = query.get_device(), query.dtype
    if query.dim() != 4 or query.shape[2] != 2:
        raise ValueError("query must be [rows, num_heads, 2, head_size]")
    rows, heads, _, size = query.shape
    n = seq_lens.shape[0]
    if out.shape != (rows, heads, 2 * size):
        raise ValueError(f"out must be {(rows, heads, 2 * size)}")
    if dtype not in _DTYPE:
        raise ValueError("query must be float32, float16 or bfloat16")
    if query_start is None:
        if rows != n:
            raise ValueError(f"query has {rows} rows for {n} sequences")
        tokens = most = 0
    else:
        if max_query_len is None:
            raise ValueError("max_query_len is required with query_start")
        tokens, most = rows, max_query_len
    if block_tables.dim() != 2 or block_tables.shape[0] != n:
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq]")
    blocks = key_cache.shape[0]
    types = (dtype,) if kv_dtype is None else _CACHE[kv_dtype]
    numel = blocks * 2 * num_kv_heads * _PAGE * size
    for name, c in (("key_cache", key_cache), ("value_cache", value_cache)):
        if c.dtype not in types:
            raise ValueError(f"{name} is {c.dtype}, kv_dtype {kv_dtype or 'same as query'} needs {types[0]}")
        if c.shape[0] != blocks or c.numel() != numel or not c.is_contiguous() or c.get_device() != device:
            raise ValueError(f"{name} must be contiguous on the call's device, {numel} elements in {blocks} pages "
                             f"(it holds {c.numel()} in {c.shape[0]})")
    stats = rows * heads * 2 * max(1, -(-max_seq_len // _abi.PA_PARTITION_SIZE))
    stride = 0
    if lambdas.dim() == 2:
        if lambdas.shape != (rows, heads) or (lambdas.stride(1) != 1 and heads > 1):
            raise ValueError("lambdas must be [num_heads] or [rows, num_heads], its heads contiguous")
        if lambdas.dtype is not torch.float32 or lambdas.get_device() != device:
            raise ValueError("lambdas must be float32 on the call's device")
        stride = lambdas.stride(0) if rows > 1 else 0
        lam = lambdas.data_ptr()
    else:
        lam = _floats("lambdas", lambdas, device, heads)
    host = None
    if seq_lens_host is not None:
        host = np.ascontiguousarray(seq_lens_host.numpy() if isinstance(seq_lens_host, torch.Tensor) else seq_lens_host,
                                    dtype=np.int32)
        if host.shape != (n,):
            raise ValueError("seq_lens_host must hold num_seqs lengths")
    return _DIFF.pack(
        _pointer("out", out, dtype, device), _pointer("query", query, dtype, device), key_cache.data_ptr(),
        value_cache.data_ptr(), _ints("block_tables", block_tables, device), _ints("seq_lens", seq_lens, device, n),
        n, heads, num_kv_heads, size, blocks, _PAGE, max_seq_len, block_tables.shape[1], scale, softcap,
        _floats("alibi_slopes", alibi_slopes, device, heads), _DTYPE[dtype], _LAYOUT[layout], _MODE[mode],
        _floats("exp_sums", exp_sums, device, stats, True), _floats("max_logits", max_logits, device, stats, True),
        _floats("tmp_out", tmp_out, device, stats * 2 * size, True), _ints("dev_error", dev_error, device, 1),
        0 if event_begin is None else event_begin.cuda_event, 0 if event_end is None else event_end.cuda_event,
        _ints("partition_counters", partition_counters, device, n * num_kv_heads, True),
        window_left + 1 if window_left >= 0 else 0, _KV[kv_dtype], k_scale, v_scale,
        _ints("query_start", query_start, device, n + 1), tokens, most,
        0 if host is None else host.__array_interface__["data"][0], _ints("tile_counters", tile_counters, device, 2),
        1 if metadata_ready else 0, 0,
        lam, stride, _floats("norm_weight", norm_weight, device, 2 * size), norm_eps, out_scale, 1 if norm else 0), host


def make_diff_args(out, query, key_cache, value_cache, block_tables, seq_lens, *, lambdas, **kw) -> _abi.PaDiffArgs:
    """Build the C argument struct of pa_diff_decode (arguments as there)."""
    packed, host = _pack_diff(out, query, key_cache, value_cache, block_tables, seq_lens, lambdas, **kw)
    args = _abi.PaDiffArgs.from_buffer_copy(packed)
    args._keep_host_lens = host  # the pointer inside stays valid as long as the struct lives
    return args


def diff_plan(args: _abi.PaDiffArgs) -> dict:
    """What pa_diff_decode would launch for a prepared struct on the current device."""
    from . import PaDecodeError
    pl = _abi.PaLaunchPlan()
    st = _abi.load().pa_diff_plan(ctypes.byref(args), ctypes.byref(pl))
    if st != _abi.PA_OK:
        raise PaDecodeError(st, "pa_diff_plan")
    return {"mode": "v1" if pl.mode == _abi.PA_MODE_V1 else "v2",
            "merge_in_kernel": bool(pl.merge_in_kernel), "kernels": int(pl.kernels),
            "ctas_per_sm": int(pl.ctas_per_sm), "grid": int(pl.grid),
            "dynamic_schedule": bool(pl.dynamic_schedule), "tiles": int(pl.tiles),
            "partition_tokens": int(pl.partition_tokens)}


def pa_diff_decode(out, query, key_cache, value_cache, block_tables, seq_lens, *, lambdas, num_kv_heads: int,
                   scale: float, max_seq_len: int, norm: bool = True, norm_weight=None, norm_eps: float = 1e-5,
                   out_scale: float = 1.0, alibi_slopes=None, softcap: float = 0.0, layout: str = "split",
                   mode: str = "auto", exp_sums=None, max_logits=None, tmp_out=None, dev_error=None,
                   event_begin=None, event_end=None, partition_counters=None, window_left: int = -1,
                   kv_dtype: str | None = None, k_scale: float = 1.0, v_scale: float = 1.0, query_start=None,
                   max_query_len: int | None = None, seq_lens_host=None, tile_counters=None,
                   metadata_ready: bool = False, stream=None) -> None:
    """Enqueue differential attention of the query rows over the paged cache.

    query [rows, num_heads, 2, head_size], out [rows, num_heads, 2 * head_size];
    key_cache with 2 * num_kv_heads heads of head_size (heads 2g and 2g + 1: the
    two maps' keys of kv head g), value_cache with num_kv_heads heads of
    2 * head_size, in the split or NHD layout; lambdas fp32 [num_heads], or [rows,
    num_heads] for a lambda per token; norm, norm_weight [2 * head_size] fp32,
    norm_eps and out_scale of the heads' RMS norm.  Everything else as pa_decode,
    with the workspace of alloc_diff_workspace (that of a larger batch or a greater
    length will do).  Rows behind query_start[num_seqs] are left as they were.  At most 8 query tokens x heads
    per kv head.  Raises PaDecodeError with the library's status on failure.
    """
    packed, _host = _pack_diff(
        out, query, key_cache, value_cache, block_tables, seq_lens, lambdas, num_kv_heads, scale, max_seq_len, norm,
        norm_weight, norm_eps, out_scale, alibi_slopes, softcap, layout, mode, exp_sums, max_logits, tmp_out, dev_error,
        event_begin, event_end, partition_counters, window_left, kv_dtype, k_scale, v_scale, query_start, max_query_len,
        seq_lens_host, tile_counters, metadata_ready)
    _call("pa_diff_decode", packed, stream, query.get_device())
