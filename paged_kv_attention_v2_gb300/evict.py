"""A cache that is short of room: Python binding of the scores, the selection and the compaction of include/pa_cache.h.

    pa_decode(out, query, key_cache, value_cache, block_tables, seq_lens, mode="v2", **ws, ...)
    pa_add_weights(scores, query, key_cache, block_tables, seq_lens, ws["exp_sums"], ws["max_logits"], ...)

after each step (with ALiBi both with relative_max=True), and when a sequence has outgrown its budget

    pa_select_tokens(kept, keep_lens, scores, block_tables, seq_lens, budgets, max_seq_len=..., sink=4, recent=64)
    pa_compact_kv(key_cache, value_cache, block_tables, kept, keep_lens, scores=scores)
    pa_build_tables(block_tables, seq_lens, ..., keep_lens=keep_lens)
"""
from __future__ import annotations

import torch

from . import _abi
from .cache import _CACHE, _DTYPE, _KV, _LAYOUT, _PAGE, _call, _ints, _pointer

_WEIGHTS = _abi.packer(_abi.PaWeightsArgs)
_SELECT = _abi.packer(_abi.PaSelectArgs)
_COMPACT = _abi.packer(_abi.PaCompactArgs)


def _floats(name: str, t, device: int, numel: int) -> int:
    return _pointer(name, t, torch.float32, device, numel)


def _check_cache(name: str, cache, types, numel: int, device: int, kv_dtype) -> None:
    if cache.dtype not in types:
        raise ValueError(f"{name} is {cache.dtype}, kv_dtype {kv_dtype or 'same as query'} needs {types[0]}")
    if cache.numel() != numel or not cache.is_contiguous() or cache.get_device() != device:
        raise ValueError(f"{name} must be contiguous, {numel} elements, on the call's device")


def _pack_weights(scores, query, key_cache, block_tables, seq_lens, exp_sums, max_logits, num_kv_heads, scale, max_seq_len,
                  decay, alibi_slopes, softcap, layout, window_left, kv_dtype, k_scale, query_start, max_query_len,
                  dev_error, relative_max) -> bytes:
    device, dtype = query.get_device(), query.dtype
    rows, heads, size = query.shape
    n = seq_lens.shape[0]
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
    _check_cache("key_cache", key_cache, (dtype,) if kv_dtype is None else _CACHE[kv_dtype],
                 blocks * num_kv_heads * size * (9 if kv_dtype == "e2m1" else _PAGE), device, kv_dtype)
    stats = rows * heads * max(1, -(-max_seq_len // _abi.PA_PARTITION_SIZE))
    return _WEIGHTS.pack(
        _floats("scores", scores, device, blocks * num_kv_heads * _PAGE), _pointer("query", query, dtype, device),
        key_cache.data_ptr(), _ints("block_tables", block_tables, device), _ints("seq_lens", seq_lens, device, n),
        _floats("exp_sums", exp_sums, device, stats), _floats("max_logits", max_logits, device, stats),
        0 if alibi_slopes is None else _floats("alibi_slopes", alibi_slopes, device, heads),
        _ints("query_start", query_start, device, n + 1), _ints("dev_error", dev_error, device, 1), n, heads, num_kv_heads,
        size, blocks, _PAGE, max_seq_len, block_tables.shape[1], tokens, most, _abi.sliding_window(window_left),
        _DTYPE[dtype], _LAYOUT[layout], _KV[kv_dtype], scale, softcap, k_scale, decay,
        1 if relative_max else 0)


def make_weights_args(scores, query, key_cache, block_tables, seq_lens, exp_sums, max_logits, *, num_kv_heads: int,
                      scale: float, max_seq_len: int, decay: float = 1.0, alibi_slopes=None, softcap: float = 0.0,
                      layout: str = "split", window_left: int = -1, kv_dtype: str | None = None, k_scale: float = 1.0,
                      query_start=None, max_query_len: int | None = None, dev_error=None,
                      relative_max: bool = False) -> _abi.PaWeightsArgs:
    """Build the C argument struct of pa_add_weights (arguments as there)."""
    return _abi.PaWeightsArgs.from_buffer_copy(
        _pack_weights(scores, query, key_cache, block_tables, seq_lens, exp_sums, max_logits, num_kv_heads, scale,
                      max_seq_len, decay, alibi_slopes, softcap, layout, window_left, kv_dtype, k_scale, query_start,
                      max_query_len, dev_error, relative_max))


def pa_add_weights(scores, query, key_cache, block_tables, seq_lens, exp_sums, max_logits, *, num_kv_heads: int,
                   scale: float, max_seq_len: int, decay: float = 1.0, alibi_slopes=None, softcap: float = 0.0,
                   layout: str = "split", window_left: int = -1, kv_dtype: str | None = None, k_scale: float = 1.0,
                   query_start=None, max_query_len: int | None = None, dev_error=None, relative_max: bool = False,
                   stream=None) -> None:
    """Add the attention weights of a decode to the score of every token it attended to.

    scores [num_blocks, num_kv_heads, 16] fp32, updated in place (decay times the old score
    plus the weights of the kv head's query heads; the step's own tokens, and with decay 0
    every token, are set); exp_sums and max_logits [rows, num_heads, partitions] as pa_decode
    left them with mode="v2" for the same query, cache and options (mode="auto" may run v1,
    which leaves them as they were: the weights would then be an earlier call's).  With
    alibi_slopes give relative_max=True to both calls: without it the weights are off by
    up to 2^-23 * slope * length.  Everything else as pa_decode; include/pa_cache.h has the formula.
    """
    args = _pack_weights(scores, query, key_cache, block_tables, seq_lens, exp_sums, max_logits, num_kv_heads, scale,
                         max_seq_len, decay, alibi_slopes, softcap, layout, window_left, kv_dtype, k_scale, query_start,
                         max_query_len, dev_error, relative_max)
    _call("pa_add_weights", args, stream, query.get_device())


def _pack_select(kept, new_seq_lens, scores, block_tables, seq_lens, budgets, max_seq_len, sink, recent, dev_error) -> bytes:
    device = seq_lens.get_device()
    if kept.dim() != 3 or block_tables.dim() != 2 or scores.dim() != 3:
        raise ValueError("kept must be [num_seqs, num_kv_heads, max_budget], block_tables [num_seqs, max_blocks_per_seq] "
                         "and scores [num_blocks, num_kv_heads, 16]")
    n, heads, most = kept.shape
    blocks = scores.shape[0]
    if block_tables.shape[0] != n:
        raise ValueError(f"{block_tables.shape[0]} rows of block_tables for {n} sequences")
    return _SELECT.pack(
        _ints("kept", kept, device), _ints("new_seq_lens", new_seq_lens, device, n),
        _floats("scores", scores, device, blocks * heads * _PAGE), _ints("block_tables", block_tables, device),
        _ints("seq_lens", seq_lens, device, n), _ints("budgets", budgets, device, n),
        _ints("dev_error", dev_error, device, 1), n, heads, blocks, _PAGE, max_seq_len, block_tables.shape[1], most, sink,
        recent)


def make_select_args(kept, new_seq_lens, scores, block_tables, seq_lens, budgets, *, max_seq_len: int, sink: int = 0,
                     recent: int = 0, dev_error=None) -> _abi.PaSelectArgs:
    """Build the C argument struct of pa_select_tokens (arguments as there)."""
    return _abi.PaSelectArgs.from_buffer_copy(
        _pack_select(kept, new_seq_lens, scores, block_tables, seq_lens, budgets, max_seq_len, sink, recent, dev_error))


def pa_select_tokens(kept, new_seq_lens, scores, block_tables, seq_lens, budgets, *, max_seq_len: int, sink: int = 0,
                     recent: int = 0, dev_error=None, stream=None) -> None:
    """Pick the tokens of each sequence that stay within its budget, for each kv head.

    kept [num_seqs, num_kv_heads, max_budget] int32 gets their positions in ascending order,
    new_seq_lens [num_seqs] int32 how many there are: min(length, budget).  The last `recent`
    tokens stay, then the first `sink`, then those with the largest scores ([num_blocks,
    num_kv_heads, 16] fp32; of equal ones the lower position).  budgets [num_seqs] int32, at
    most max_budget each.
    """
    args = _pack_select(kept, new_seq_lens, scores, block_tables, seq_lens, budgets, max_seq_len, sink, recent, dev_error)
    _call("pa_select_tokens", args, stream, seq_lens.get_device())


_BY_TYPE = {torch.float32: _abi.PA_DTYPE_F32, torch.float16: _abi.PA_DTYPE_F16, torch.bfloat16: _abi.PA_DTYPE_BF16}


def _head_size(name: str, cache, layout: str, kv_dtype, is_key: bool) -> int:
    if kv_dtype == "e2m1":
        if cache.dim() != 3 or cache.shape[2] % 9:
            raise ValueError(f"{name} must be [num_blocks, heads, 9 * head size]")
        return cache.shape[2] // 9
    if layout == "nhd":
        if cache.dim() != 4 or cache.shape[2] != _PAGE:
            raise ValueError(f"{name} must be [num_blocks, heads, 16, head size]")
        return cache.shape[3]
    if is_key:
        if cache.dim() != 5 or cache.shape[3] != _PAGE or cache.shape[4] * cache.element_size() != 16:
            raise ValueError(f"{name} must be [num_blocks, heads, head size / x, 16, x], 16 bytes of x")
        return cache.shape[2] * cache.shape[4]
    if cache.dim() != 4 or cache.shape[3] != _PAGE:
        raise ValueError(f"{name} must be [num_blocks, heads, head size, 16]")
    return cache.shape[2]


def _pack_compact(key_cache, value_cache, block_tables, kept, new_seq_lens, scores, layout, kv_dtype, dev_error) -> bytes:
    device = kept.get_device()
    if kept.dim() != 3 or block_tables.dim() != 2:
        raise ValueError("kept must be [num_seqs, num_kv_heads, max_budget] and block_tables [num_seqs, max_blocks_per_seq]")
    n, heads, most = kept.shape
    blocks = key_cache.shape[0]
    if block_tables.shape[0] != n:
        raise ValueError(f"{block_tables.shape[0]} rows of block_tables for {n} sequences")
    if value_cache.shape[0] != blocks:
        raise ValueError(f"{blocks} key pages and {value_cache.shape[0]} value pages")
    types = tuple(_BY_TYPE) if kv_dtype is None else _CACHE[kv_dtype]
    if value_cache.dtype is not key_cache.dtype:
        raise ValueError("key_cache and value_cache must be of one type")
    sizes = []
    for name, cache in (("key_cache", key_cache), ("value_cache", value_cache)):
        _check_cache(name, cache, types, cache.numel(), device, kv_dtype)
        sizes.append(_head_size(name, cache, layout, kv_dtype, name == "key_cache"))
    return _COMPACT.pack(
        key_cache.data_ptr(), value_cache.data_ptr(),
        0 if scores is None else _floats("scores", scores, device, blocks * heads * _PAGE),
        _ints("block_tables", block_tables, device), _ints("kept", kept, device),
        _ints("new_seq_lens", new_seq_lens, device, n), _ints("dev_error", dev_error, device, 1), n, heads, most,
        key_cache.shape[1], sizes[0], value_cache.shape[1], sizes[1], blocks, _PAGE, block_tables.shape[1],
        _abi.PA_DTYPE_F16 if kv_dtype is not None else _BY_TYPE[key_cache.dtype], _LAYOUT[layout], _KV[kv_dtype])


def make_compact_args(key_cache, value_cache, block_tables, kept, new_seq_lens, *, scores=None, layout: str = "split",
                      kv_dtype: str | None = None, dev_error=None) -> _abi.PaCompactArgs:
    """Build the C argument struct of pa_compact_kv (arguments as there)."""
    return _abi.PaCompactArgs.from_buffer_copy(
        _pack_compact(key_cache, value_cache, block_tables, kept, new_seq_lens, scores, layout, kv_dtype, dev_error))


def pa_compact_kv(key_cache, value_cache, block_tables, kept, new_seq_lens, *, scores=None, layout: str = "split",
                  kv_dtype: str | None = None, dev_error=None, stream=None) -> None:
    """Move the tokens that stay to the front of their sequence's pages, in place.

    kept [num_seqs, num_kv_heads, max_budget] and new_seq_lens [num_seqs] int32 as from
    pa_select_tokens (positions ascend in each row): token kept[s, h, i] becomes token i, keys,
    values and, given, scores.  Caches in the shapes of include/pa_decode.h, with head counts that are
    multiples of num_kv_heads (a differential cache has two key heads to each value head).
    """
    args = _pack_compact(key_cache, value_cache, block_tables, kept, new_seq_lens, scores, layout, kv_dtype, dev_error)
    _call("pa_compact_kv", args, stream, kept.get_device())
