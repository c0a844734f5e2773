"""The paged cache between decode steps: Python binding of include/pa_cache.h.

    pa_build_tables(block_tables, seq_lens, free_ring, pool_state, slots, max_seq_len=...)
    pa_append_kv(key, value, key_cache, value_cache, slots, layout="split")
    pa_decode(out, query, key_cache, value_cache, block_tables, seq_lens, ...)

is one step of serving: the lengths, the tables and the pool move on in place.
"""
from __future__ import annotations

import torch

from . import _abi

_LAYOUT = {"split": _abi.PA_LAYOUT_SPLIT, "nhd": _abi.PA_LAYOUT_NHD}
_KV = {None: _abi.PA_KV_SAME, "e4m3": _abi.PA_KV_FP8_E4M3, "e5m2": _abi.PA_KV_FP8_E5M2}
_DTYPE = {torch.float32: _abi.PA_DTYPE_F32, torch.float16: _abi.PA_DTYPE_F16,
          torch.bfloat16: _abi.PA_DTYPE_BF16}
# cache element types of each kv_dtype (None: the rows' own)
_CACHE = {"e4m3": (torch.uint8, torch.float8_e4m3fn), "e5m2": (torch.uint8, torch.float8_e5m2)}
_TABLES = _abi.packer(_abi.PaTablesArgs)
_APPEND = _abi.packer(_abi.PaAppendArgs)
_PAGE = _abi.PA_BLOCK_SIZE


def _call(name: str, args: bytes, stream, device: int) -> None:
    """The entry point `name` with packed arguments on `stream` (default: torch's
    current one), with the tensors' device current."""
    if device < 0:
        raise ValueError(f"{name} needs CUDA tensors")
    fn = getattr(_abi.load(), name)
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device)
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if torch.cuda.current_device() == device:
        st = fn(args, handle)
    else:
        with torch.cuda.device(device):
            st = fn(args, handle)
    if st != _abi.PA_OK:
        from . import PaDecodeError
        raise PaDecodeError(st, name)


def _pointer(name: str, t, dtype, device: int, numel: int = -1, room: bool = False) -> int:
    """Address of a contiguous tensor of `dtype` on `device` (None: 0), of `numel`
    elements if given (with `room` at least as many)."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on the call's device")
    if numel >= 0 and t.numel() != numel and not (room and t.numel() > numel):
        raise ValueError(f"{name} holds {t.numel()} elements, expected {'at least ' if room else ''}{numel}")
    return t.data_ptr()


def _ints(name: str, t, device: int, numel: int = -1, room: bool = False) -> int:
    return _pointer(name, t, torch.int32, device, numel, room)


def _pack_tables(block_tables, seq_lens, free_ring, pool_state, slots, max_seq_len, keep_lens, query_start,
                 positions, new_seq_lens, new_pool_state, done_counter, dev_error) -> bytes:
    device = seq_lens.get_device()
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq]")
    n, width = block_tables.shape
    rows = slots.numel()
    lens = _ints("seq_lens", seq_lens, device, n)
    state = _ints("pool_state", pool_state, device, 2)
    return _TABLES.pack(
        _ints("block_tables", block_tables, device), lens, _ints("keep_lens", keep_lens, device, n),
        _ints("query_start", query_start, device, n + 1), _ints("free_ring", free_ring, device), state,
        _ints("slots", slots, device), _ints("positions", positions, device, rows),
        lens if new_seq_lens is None else _ints("new_seq_lens", new_seq_lens, device, n),
        state if new_pool_state is None else _ints("new_pool_state", new_pool_state, device, 2),
        n, rows, free_ring.numel(), _PAGE, max_seq_len, width, _ints("dev_error", dev_error, device, 1),
        _ints("done_counter", done_counter, device, 1))


def make_tables_args(block_tables, seq_lens, free_ring, pool_state, slots, *, max_seq_len: int,
                     keep_lens=None, query_start=None, positions=None, new_seq_lens=None,
                     new_pool_state=None, done_counter=None, dev_error=None) -> _abi.PaTablesArgs:
    """Build the C argument struct of pa_build_tables (arguments as there)."""
    return _abi.PaTablesArgs.from_buffer_copy(
        _pack_tables(block_tables, seq_lens, free_ring, pool_state, slots, max_seq_len, keep_lens, query_start,
                     positions, new_seq_lens, new_pool_state, done_counter, dev_error))


def pa_build_tables(block_tables, seq_lens, free_ring, pool_state, slots, *, max_seq_len: int,
                    keep_lens=None, query_start=None, positions=None, new_seq_lens=None,
                    new_pool_state=None, done_counter=None, dev_error=None, stream=None) -> None:
    """Hand out pages for a step's tokens and map them to cache slots, on the GPU.

    Contiguous int32 CUDA tensors: block_tables [num_seqs, max_blocks_per_seq] and
    free_ring [num_blocks] are updated in place; seq_lens [num_seqs] are the tokens
    stored so far and pool_state [2] the ring's {head, count}; new_seq_lens and
    new_pool_state get the values after the step (default: over the old ones).
    query_start [num_seqs + 1] gives each sequence's new tokens (one each without
    it), keep_lens [num_seqs] the tokens that stay (all without it; 0 ends a
    sequence).  slots [rows] and positions [rows] (optional) are written for every
    row, -1 and 0 behind the last token.  done_counter [1] (int32, zeroed once)
    lets a call of many rows use the whole GPU (2.1 million rows: 8.6 us, 429 without).
    Everything else, and what happens when the pool runs short, is in include/pa_cache.h.
    """
    args = _pack_tables(block_tables, seq_lens, free_ring, pool_state, slots, max_seq_len, keep_lens, query_start,
                        positions, new_seq_lens, new_pool_state, done_counter, dev_error)
    _call("pa_build_tables", args, stream, seq_lens.get_device())


def _pack_append(key, value, key_cache, value_cache, slots, layout, kv_dtype, k_scale, v_scale, dev_error) -> bytes:
    device, dtype = key.get_device(), key.dtype
    tokens, k_heads, k_size = key.shape
    v_tokens, v_heads, v_size = value.shape
    if v_tokens != tokens:
        raise ValueError(f"{tokens} keys and {v_tokens} values")
    if value.dtype is not dtype or dtype not in _DTYPE:
        raise ValueError("key and value must both be float32, float16 or bfloat16")
    types = (dtype,) if kv_dtype is None else _CACHE[kv_dtype]
    blocks = key_cache.shape[0]
    if value_cache.shape[0] != blocks:
        raise ValueError(f"{blocks} key pages and {value_cache.shape[0]} value pages")
    ks, kh, kd = key.stride()
    vs, vh, vd = value.stride()
    if kd != 1 or vd != 1:
        raise ValueError("the head dims of key and value must be contiguous")
    if value.get_device() != device:
        raise ValueError("key and value must be on one device")
    for name, cache, page in (("key_cache", key_cache, k_heads * k_size * _PAGE),
                              ("value_cache", value_cache, v_heads * v_size * _PAGE)):
        if cache.dtype not in types:
            raise ValueError(f"{name} is {cache.dtype}, kv_dtype {kv_dtype or 'same as key'} needs {types[0]}")
        if cache.numel() != blocks * page or not cache.is_contiguous() or cache.get_device() != device:
            raise ValueError(f"{name} must be contiguous, {blocks} pages of {page} elements, on the call's device")
    # the stride of a dimension of one is never used
    if tokens <= 1:
        ks = vs = 0
    return _APPEND.pack(
        key.data_ptr(), value.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
        _ints("slots", slots, device, tokens), ks, kh if k_heads > 1 else 0, vs, vh if v_heads > 1 else 0, tokens,
        k_heads, k_size, v_heads, v_size, blocks, _PAGE, _DTYPE[dtype], _LAYOUT[layout], _KV[kv_dtype], k_scale,
        v_scale, _ints("dev_error", dev_error, device, 1))


def make_append_args(key, value, key_cache, value_cache, slots, *, layout: str = "split",
                     kv_dtype: str | None = None, k_scale: float = 1.0, v_scale: float = 1.0,
                     dev_error=None) -> _abi.PaAppendArgs:
    """Build the C argument struct of pa_append_kv (arguments as there)."""
    return _abi.PaAppendArgs.from_buffer_copy(
        _pack_append(key, value, key_cache, value_cache, slots, layout, kv_dtype, k_scale, v_scale, dev_error))


def pa_append_kv(key, value, key_cache, value_cache, slots, *, layout: str = "split",
                 kv_dtype: str | None = None, k_scale: float = 1.0, v_scale: float = 1.0,
                 dev_error=None, stream=None) -> None:
    """Store the keys and values of a step's tokens into the paged cache.

    key [tokens, key heads, key head size] and value [tokens, value heads, value
    head size] (fp32, fp16 or bf16; token and head strides may be anything that is
    a multiple of 16 bytes, as in a slice of a fused projection), slots [tokens]
    int32 from pa_build_tables (negative: skip), caches in the split or NHD
    layout; kv_dtype "e4m3" / "e5m2" quantises to fp8 caches (torch's fp8 types or
    raw uint8) holding K / k_scale and V / v_scale (the fp32 quotients, rounded).
    """
    args = _pack_append(key, value, key_cache, value_cache, slots, layout, kv_dtype, k_scale, v_scale, dev_error)
    _call("pa_append_kv", args, stream, key.get_device())
