"""Host-side checks of pa_build_tables and pa_append_kv (no GPU): the argument
structs match the header, and every refusal comes before anything is launched."""
import ctypes
import pathlib
import shutil
import subprocess

import numpy as np
import pytest

import paged_kv_attention_v2_gb300 as pa
from cache_ref import make_batch, tables_ref
from paged_kv_attention_v2_gb300 import _abi, cache

INC = pathlib.Path(__file__).resolve().parents[1] / "include"


@pytest.fixture(scope="module")
def lib():
    from paged_kv_attention_v2_gb300 import build
    build.build()
    return _abi.load()


def test_struct_layouts_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    pairs = (("pa_tables_args", _abi.PaTablesArgs), ("pa_append_args", _abi.PaAppendArgs))
    lines = ['#include <stdio.h>', '#include "pa_cache.h"', "int main(void) {"]
    for cname, cls in pairs:
        lines.append(f'printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0;", "}"]) + "\n")
    subprocess.run([cc, "-std=c11", "-I", str(INC), str(src), "-o", str(tmp_path / "layout")], check=True)
    out = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout
    got = {tuple(line.split()[:2]): int(line.split()[2]) for line in out.splitlines()}
    for cname, cls in pairs:
        assert got[(cname, "size")] == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert got[(cname, f)] == getattr(cls, f).offset, (cname, f)


def _tables(**over):
    a = _abi.PaTablesArgs(
        block_tables=16, seq_lens=16, free_ring=16, pool_state=16, slots=16, positions=16, new_seq_lens=16,
        new_pool_state=16, num_seqs=4, num_tokens=4, num_blocks=100, block_size=16, max_seq_len=100,
        max_blocks_per_seq=7)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,expect", [
    ({"num_seqs": -1}, _abi.PA_ERR_INVALID_ARG),
    ({"num_tokens": -1}, _abi.PA_ERR_INVALID_ARG),
    ({"num_tokens": 3}, _abi.PA_ERR_INVALID_ARG),            # one token each, three rows
    ({"num_blocks": 0}, _abi.PA_ERR_INVALID_ARG),
    ({"num_blocks": 1 << 27}, _abi.PA_ERR_UNSUPPORTED),      # slots would pass 31 bits
    ({"block_size": 32}, _abi.PA_ERR_UNSUPPORTED),
    ({"max_blocks_per_seq": 6}, _abi.PA_ERR_INVALID_ARG),
    ({"max_seq_len": -1}, _abi.PA_ERR_INVALID_ARG),
    ({"num_seqs": 1 << 20, "num_tokens": 1 << 20, "max_blocks_per_seq": 1 << 11}, _abi.PA_ERR_UNSUPPORTED),
    ({"num_tokens": (1 << 30) + 1}, _abi.PA_ERR_UNSUPPORTED),   # counted in 32 bits
    ({"num_seqs": (1 << 30) + 1, "num_tokens": 1 << 30, "query_start": 16, "max_seq_len": 0, "max_blocks_per_seq": 1},
     _abi.PA_ERR_UNSUPPORTED),
    ({"block_tables": None}, _abi.PA_ERR_INVALID_ARG),
    ({"seq_lens": None}, _abi.PA_ERR_INVALID_ARG),
    ({"free_ring": None}, _abi.PA_ERR_INVALID_ARG),
    ({"pool_state": None}, _abi.PA_ERR_INVALID_ARG),
    ({"slots": None}, _abi.PA_ERR_INVALID_ARG),
    ({"new_seq_lens": None}, _abi.PA_ERR_INVALID_ARG),
    ({"new_pool_state": None}, _abi.PA_ERR_INVALID_ARG),
    ({"slots": 18}, _abi.PA_ERR_INVALID_ARG),
    ({"done_counter": 2}, _abi.PA_ERR_INVALID_ARG),
])
def test_tables_refusals(lib, over, expect):
    assert lib.pa_build_tables(ctypes.byref(_tables(**over)), None) == expect


def _append(**over):
    a = _abi.PaAppendArgs(
        key=16, value=16, key_cache=16, value_cache=16, slots=16, key_stride=256, key_head_stride=128,
        value_stride=256, value_head_stride=128, num_tokens=3, num_key_heads=2, key_head_size=128, num_value_heads=2,
        value_head_size=128, num_blocks=10, block_size=16, dtype=_abi.PA_DTYPE_F16, layout=_abi.PA_LAYOUT_NHD,
        kv_dtype=_abi.PA_KV_SAME, k_scale=1.0, v_scale=1.0)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,expect", [
    ({"num_tokens": -1}, _abi.PA_ERR_INVALID_ARG),
    ({"num_key_heads": 0}, _abi.PA_ERR_INVALID_ARG),
    ({"num_value_heads": 0}, _abi.PA_ERR_INVALID_ARG),
    ({"num_key_heads": 40000, "num_value_heads": 40000}, _abi.PA_ERR_UNSUPPORTED),
    ({"key_head_size": 96}, _abi.PA_ERR_UNSUPPORTED),
    ({"value_head_size": 512}, _abi.PA_ERR_UNSUPPORTED),
    ({"num_blocks": 0}, _abi.PA_ERR_INVALID_ARG),
    ({"num_blocks": 1 << 27}, _abi.PA_ERR_UNSUPPORTED),
    ({"block_size": 8}, _abi.PA_ERR_UNSUPPORTED),
    ({"dtype": 5}, _abi.PA_ERR_INVALID_ARG),
    ({"layout": 2}, _abi.PA_ERR_INVALID_ARG),
    ({"kv_dtype": 1}, _abi.PA_ERR_INVALID_ARG),
    ({"kv_dtype": _abi.PA_KV_FP8_E4M3, "dtype": _abi.PA_DTYPE_F32}, _abi.PA_ERR_UNSUPPORTED),
    ({"k_scale": float("nan")}, _abi.PA_ERR_INVALID_ARG),
    ({"v_scale": 1e-40}, _abi.PA_ERR_INVALID_ARG),
    ({"key": None}, _abi.PA_ERR_INVALID_ARG),
    ({"slots": None}, _abi.PA_ERR_INVALID_ARG),
    ({"value": 8}, _abi.PA_ERR_INVALID_ARG),
    ({"key_cache": 8}, _abi.PA_ERR_INVALID_ARG),
    ({"key_stride": 257}, _abi.PA_ERR_INVALID_ARG),
    ({"value_head_stride": 4}, _abi.PA_ERR_INVALID_ARG),
    ({"num_tokens": (1 << 30) + 1}, _abi.PA_ERR_UNSUPPORTED),
    ({"num_tokens": 0, "key": None}, _abi.PA_OK),
])
def test_append_refusals(lib, over, expect):
    assert lib.pa_append_kv(ctypes.byref(_append(**over)), None) == expect


def test_null_args(lib):
    assert lib.pa_build_tables(None, None) == _abi.PA_ERR_INVALID_ARG
    assert lib.pa_append_kv(None, None) == _abi.PA_ERR_INVALID_ARG


def test_binding_refuses_what_only_the_tensors_know():
    import torch
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    ok = dict(block_tables=i(3, 4), seq_lens=i(3), free_ring=i(9), pool_state=i(2), slots=i(3))
    kw = dict(max_seq_len=64)
    cache.make_tables_args(**ok, **kw)
    with pytest.raises(ValueError):
        pa.pa_build_tables(*ok.values(), **kw)                                   # not on a GPU
    for bad in (dict(seq_lens=i(2)), dict(slots=torch.zeros(3, dtype=torch.int64)), dict(pool_state=i(3)),
                dict(block_tables=i(4, 3).t()), dict(block_tables=i(12))):
        with pytest.raises(ValueError):
            cache.make_tables_args(**{**ok, **bad}, **kw)
    for bad in (dict(keep_lens=i(2)), dict(query_start=i(3)), dict(positions=i(4)), dict(new_seq_lens=i(4)),
                dict(done_counter=i(2))):
        with pytest.raises(ValueError):
            cache.make_tables_args(**ok, **kw, **bad)

    h = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    good = (h(5, 2, 64), h(5, 2, 64), h(7, 2, 16, 64), h(7, 2, 16, 64), i(5))
    cache.make_append_args(*good, layout="nhd")
    with pytest.raises(ValueError):
        pa.pa_append_kv(*good, layout="nhd")                                     # not on a GPU
    for at, bad in ((1, h(4, 2, 64)), (1, h(5, 2, 64).float()), (2, h(7, 2, 16, 128)), (3, h(6, 2, 16, 64)),
                    (2, h(7, 2, 64, 16).transpose(2, 3)), (3, h(7, 2, 16, 64).bfloat16()), (4, i(4)), (0, h(5, 64, 2).transpose(1, 2))):
        with pytest.raises(ValueError):
            cache.make_append_args(*good[:at], bad, *good[at + 1:], layout="nhd")
    with pytest.raises(ValueError):
        cache.make_append_args(*good, layout="nhd", kv_dtype="e4m3")             # 2-byte caches
    fp8 = [torch.zeros((7, 2, 16, 64), dtype=t) for t in (torch.uint8, torch.float8_e4m3fn, torch.float8_e5m2)]
    for c in fp8[:2]:
        cache.make_append_args(*good[:2], c, c, good[4], layout="nhd", kv_dtype="e4m3")
    with pytest.raises(ValueError):
        cache.make_append_args(*good[:2], fp8[2], fp8[2], good[4], layout="nhd", kv_dtype="e4m3")
    # one row: its strides are never used, whatever they are
    odd = torch.as_strided(h(200), (1, 1, 64), (3, 5, 1))
    a = cache.make_append_args(odd, odd, h(7, 1, 16, 64), h(7, 1, 16, 64), i(1), layout="nhd")
    assert (a.key_stride, a.key_head_stride, a.value_stride, a.value_head_stride) == (0, 0, 0, 0)


def test_reference_keeps_every_page_in_one_place():
    """The plain statement itself: after a step every page is owned once or free once."""
    b = make_batch(3, 20, 300, 30, cut=True)
    table, ring, slots, positions, new, state = tables_ref(b["table"], b["lens"], b["ring"], b["state"],
                                                           b["tokens"], b["keep"], b["start"])
    owned = [table[s, p] for s in range(20) for p in range(-(-int(new[s]) // 16))]
    free = [ring[(state[0] + k) % len(ring)] for k in range(state[1])]
    assert sorted(owned + free) == list(range(len(ring)))
    assert len(set(slots)) == b["tokens"] and np.all(slots >= 0)
