"""Host-side checks (no GPU) of 4-bit caches, pa_add_weights, pa_select_tokens and
pa_compact_kv: the structs match the header, refusals come before anything is launched, and the
plain statements that the GPU tests compare with are themselves compared with loops."""
import ctypes
import pathlib
import shutil
import subprocess
from fractions import Fraction

import numpy as np
import pytest

import paged_kv_attention_v2_gb300 as pa
from paged_kv_attention_v2_gb300 import _abi, cache, evict
from short_ref import compact_ref, e4m3_values, pages4, quantise4, select_ref, store4, values4

torch = pytest.importorskip("torch")
INC = pathlib.Path(__file__).resolve().parents[1] / "include"
OK, BAD, NO = _abi.PA_OK, _abi.PA_ERR_INVALID_ARG, _abi.PA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from paged_kv_attention_v2_gb300 import build
    build.build()
    return _abi.load()


def test_struct_layouts_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    pairs = (("pa_weights_args", _abi.PaWeightsArgs), ("pa_select_args", _abi.PaSelectArgs), ("pa_compact_args", _abi.PaCompactArgs))
    lines = ['#include <stdio.h>', '#include "pa_cache.h"', "int main(void) {", 'printf("kv fp4 %d\\n", PA_KV_FP4_E2M1);']
    for cname, cls in pairs:
        lines.append(f'printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0;", "}"]) + "\n")
    subprocess.run([cc, "-std=c11", "-I", str(INC), str(src), "-o", str(tmp_path / "layout")], check=True)
    out = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout
    got = {tuple(line.split()[:2]): int(line.split()[2]) for line in out.splitlines()}
    assert got[("kv", "fp4")] == _abi.PA_KV_FP4_E2M1
    for cname, cls in pairs:
        assert got[(cname, "size")] == ctypes.sizeof(cls) == _abi.packer(cls).size
        for f, _ in cls._fields_:
            assert got[(cname, f)] == getattr(cls, f).offset, (cname, f)


def _with(a, over):
    for k, v in over.items():
        setattr(a, k, v)
    return a


def _append(**over):
    return _with(_abi.PaAppendArgs(
        key=16, value=16, key_cache=16, value_cache=16, slots=16, key_stride=256, key_head_stride=128, value_stride=256,
        value_head_stride=128, num_tokens=3, num_key_heads=2, key_head_size=128, num_value_heads=2, value_head_size=128,
        num_blocks=10, block_size=16, dtype=_abi.PA_DTYPE_F16, layout=_abi.PA_LAYOUT_NHD, kv_dtype=_abi.PA_KV_FP4_E2M1,
        k_scale=1.0, v_scale=1.0), over)


@pytest.mark.parametrize("over,expect", [
    ({"dtype": _abi.PA_DTYPE_F32}, NO),
    ({"layout": _abi.PA_LAYOUT_SPLIT}, NO),
    ({"key_head_size": 256}, NO),
    ({"value_head_size": 256}, NO),
    ({"kv_dtype": 6}, BAD),
    ({"k_scale": float("inf")}, BAD),
    ({"v_scale": 1e-40}, BAD),
    ({"key_stride": 4}, BAD),
    ({"value_cache": 24}, BAD),
    ({"num_tokens": 0, "key": None}, OK),
    ({"num_tokens": 0, "layout": _abi.PA_LAYOUT_SPLIT}, NO),
])
def test_append_refusals(lib, over, expect):
    assert lib.pa_append_kv(ctypes.byref(_append(**over)), None) == expect


def _decode(**over):
    return _with(_abi.PaDecodeArgs(
        out=16, query=16, key_cache=16, value_cache=16, block_tables=16, seq_lens=16, num_seqs=2, num_heads=8, num_kv_heads=2,
        head_size=64, num_blocks=10, block_size=16, max_seq_len=100, max_blocks_per_seq=7, scale=0.1, dtype=_abi.PA_DTYPE_F16,
        layout=_abi.PA_LAYOUT_NHD, mode=_abi.PA_MODE_V2, kv_dtype=_abi.PA_KV_FP4_E2M1), over)


@pytest.mark.parametrize("over,expect", [
    ({"dtype": _abi.PA_DTYPE_F32}, NO),
    ({"layout": _abi.PA_LAYOUT_SPLIT}, NO),
    ({"kv_dtype": 6}, BAD),
    ({"head_size": 256}, NO),
    ({}, _abi.PA_ERR_WORKSPACE),
    ({"num_seqs": 0}, OK),
])
def test_decode_refusals(lib, over, expect):
    assert lib.pa_decode(ctypes.byref(_decode(**over)), None) == expect


def test_differential_caches_are_not_held_in_four_bits(lib):
    a = _abi.PaDiffArgs(_decode(exp_sums=16, max_logits=16, tmp_out=16), 16, 0, None, 1e-5, 1.0, 1)
    assert lib.pa_diff_decode(ctypes.byref(a), None) == NO


def _weights(**over):
    return _with(_abi.PaWeightsArgs(
        scores=16, query=16, key_cache=16, block_tables=16, seq_lens=16, exp_sums=16, max_logits=16, num_seqs=2, num_heads=8,
        num_kv_heads=2, head_size=64, num_blocks=10, block_size=16, max_seq_len=100, max_blocks_per_seq=7,
        dtype=_abi.PA_DTYPE_F16, layout=_abi.PA_LAYOUT_NHD, kv_dtype=_abi.PA_KV_SAME, scale=0.1, k_scale=1.0, decay=1.0), over)


@pytest.mark.parametrize("over,expect", [
    ({"num_heads": 7}, BAD), ({"num_heads": 0}, BAD), ({"num_seqs": -1}, BAD), ({"num_blocks": 0}, BAD),
    ({"num_heads": 34}, NO),                                          # 17 rows to a kv head
    ({"query_start": 16, "max_query_len": 5, "num_query_tokens": 4}, NO),
    ({"query_start": 16, "max_query_len": 0}, BAD), ({"query_start": 18, "max_query_len": 1}, BAD),
    ({"head_size": 256}, NO), ({"block_size": 32}, NO), ({"max_seq_len": (1 << 30) + 1, "max_blocks_per_seq": 1 << 27}, NO),
    ({"max_blocks_per_seq": 6}, BAD), ({"dtype": 3}, BAD), ({"layout": 2}, BAD), ({"kv_dtype": 2}, BAD),
    ({"kv_dtype": _abi.PA_KV_FP4_E2M1, "layout": _abi.PA_LAYOUT_SPLIT}, NO), ({"kv_dtype": _abi.PA_KV_FP8_E4M3, "dtype": 0}, NO),
    ({"decay": -0.5}, BAD), ({"decay": float("nan")}, BAD), ({"scale": float("inf")}, BAD), ({"softcap": float("nan")}, BAD),
    ({"scores": None}, BAD), ({"query": None}, BAD), ({"exp_sums": None}, BAD), ({"max_logits": None}, BAD), ({"query": 8}, BAD),
    ({"scores": 18}, BAD), ({"num_seqs": 0, "scores": None}, OK), ({"max_seq_len": 0, "query": None}, OK),
])
def test_weights_refusals(lib, over, expect):
    assert lib.pa_add_weights(ctypes.byref(_weights(**over)), None) == expect


def _select(**over):
    return _with(_abi.PaSelectArgs(
        kept=16, new_seq_lens=32, scores=16, block_tables=16, seq_lens=16, budgets=16, num_seqs=2, num_kv_heads=2, num_blocks=10,
        block_size=16, max_seq_len=100, max_blocks_per_seq=7, max_budget=50), over)


@pytest.mark.parametrize("over,expect", [
    ({"num_seqs": -1}, BAD), ({"num_kv_heads": 0}, BAD), ({"num_blocks": 0}, BAD), ({"max_budget": -1}, BAD), ({"sink": -1}, BAD),
    ({"recent": -1}, BAD), ({"block_size": 8}, NO), ({"max_seq_len": (1 << 30) + 1, "max_blocks_per_seq": 1 << 27}, NO),
    ({"max_budget": (1 << 30) + 1}, NO), ({"num_seqs": 1 << 28}, NO), ({"kept": None}, BAD), ({"scores": None}, BAD),
    ({"budgets": None}, BAD), ({"new_seq_lens": 16}, BAD),            # the lengths themselves
    ({"max_blocks_per_seq": 6}, BAD), ({"kept": 18}, BAD), ({"scores": 24}, BAD),
    ({"num_seqs": 0, "kept": None}, OK),
])
def test_select_refusals(lib, over, expect):
    assert lib.pa_select_tokens(ctypes.byref(_select(**over)), None) == expect


def _compact(**over):
    return _with(_abi.PaCompactArgs(
        key_cache=16, value_cache=16, scores=16, block_tables=16, kept=16, new_seq_lens=16, num_seqs=2, num_kv_heads=2,
        max_budget=50, num_key_heads=4, key_head_size=64, num_value_heads=2, value_head_size=128, num_blocks=10, block_size=16,
        max_blocks_per_seq=7, dtype=_abi.PA_DTYPE_F16, layout=_abi.PA_LAYOUT_SPLIT, kv_dtype=_abi.PA_KV_SAME), over)


@pytest.mark.parametrize("over,expect", [
    ({"num_key_heads": 3}, BAD), ({"num_value_heads": 1}, BAD), ({"num_kv_heads": 0}, BAD), ({"max_budget": 113}, BAD),
    ({"max_budget": -1}, BAD), ({"key_head_size": 96}, NO), ({"value_head_size": 512}, NO), ({"block_size": 8}, NO),
    ({"num_blocks": 1 << 27}, NO), ({"dtype": 4}, BAD), ({"layout": 3}, BAD), ({"kv_dtype": 1}, BAD),
    ({"kv_dtype": _abi.PA_KV_FP4_E2M1}, NO), ({"kv_dtype": _abi.PA_KV_FP4_E2M1, "layout": 1, "value_head_size": 256}, NO),
    ({"kv_dtype": _abi.PA_KV_FP8_E5M2, "dtype": 0}, NO), ({"key_cache": None}, BAD), ({"value_cache": 8}, BAD), ({"kept": None}, BAD),
    ({"scores": 2}, BAD), ({"num_key_heads": 65538}, NO), ({"num_seqs": 0, "kept": None}, OK), ({"max_budget": 0, "kept": None}, OK),
    ({"max_budget": (1 << 30) + 1, "max_blocks_per_seq": (1 << 27) - 1}, NO),
])
def test_compact_refusals(lib, over, expect):
    assert lib.pa_compact_kv(ctypes.byref(_compact(**over)), None) == expect


def test_null_args(lib):
    for fn in (lib.pa_add_weights, lib.pa_select_tokens, lib.pa_compact_kv):
        assert fn(None, None) == BAD


def test_binding_refuses_what_only_the_tensors_know():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    h = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    f = lambda *s: torch.zeros(s)  # noqa: E731
    b = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    # 4-bit append and decode
    rows = (h(5, 2, 64), h(5, 2, 64))
    cache.make_append_args(*rows, b(7, 2, 576), b(7, 2, 576), i(5), layout="nhd", kv_dtype="e2m1")
    for k, v in ((b(7, 2, 512), b(7, 2, 576)), (b(7, 2, 576), h(7, 2, 576)), (b(7, 2, 16, 64), b(7, 2, 16, 64))):
        with pytest.raises(ValueError):
            cache.make_append_args(*rows, k, v, i(5), layout="nhd", kv_dtype="e2m1")
    kw = dict(num_kv_heads=2, scale=0.1, max_seq_len=40, layout="nhd", kv_dtype="e2m1")
    pa.make_args(h(3, 4, 64), h(3, 4, 64), b(7, 2, 576), b(7, 2, 576), i(3, 3), i(3), **kw)
    with pytest.raises(ValueError):
        pa.make_args(h(3, 4, 64), h(3, 4, 64), b(7, 2, 16, 64), b(7, 2, 16, 64), i(3, 3), i(3), **kw)
    with pytest.raises(ValueError):
        pa.pa_decode(h(3, 4, 64), h(3, 4, 64), b(7, 2, 576), b(7, 2, 576), i(3, 3), i(3), **kw)   # not on a GPU
    # weights
    good = dict(scores=f(7, 2, 16), query=h(3, 4, 64), key_cache=h(7, 2, 16, 64), block_tables=i(3, 3), seq_lens=i(3),
                exp_sums=f(3, 4, 1), max_logits=f(3, 4, 1))
    kw = dict(num_kv_heads=2, scale=0.1, max_seq_len=40, layout="nhd")
    evict.make_weights_args(**good, **kw)
    with pytest.raises(ValueError):
        pa.pa_add_weights(**good, **kw)                                                          # not on a GPU
    for bad in (dict(scores=f(7, 2, 15)), dict(scores=h(7, 2, 16)), dict(query=h(4, 4, 64)), dict(key_cache=h(7, 2, 16, 32)),
                dict(key_cache=f(7, 2, 16, 64)), dict(block_tables=i(2, 3)), dict(exp_sums=f(3, 4, 2)), dict(max_logits=f(3, 2, 1)),
                dict(seq_lens=torch.zeros(3, dtype=torch.int64)), dict(query=torch.zeros(3, 4, 64, dtype=torch.float64))):
        with pytest.raises(ValueError):
            evict.make_weights_args(**{**good, **bad}, **kw)
    with pytest.raises(ValueError):
        evict.make_weights_args(**good, **kw, query_start=i(4))                                  # no max_query_len
    # selection
    good = dict(kept=i(3, 2, 30), new_seq_lens=i(3), scores=f(7, 2, 16), block_tables=i(3, 3), seq_lens=i(3), budgets=i(3))
    evict.make_select_args(**good, max_seq_len=40)
    for bad in (dict(kept=i(3, 60)), dict(kept=i(3, 3, 30)), dict(new_seq_lens=i(2)), dict(scores=f(7, 32)), dict(block_tables=i(4, 3)),
                dict(budgets=f(3)), dict(kept=i(3, 30, 2).transpose(1, 2))):
        with pytest.raises(ValueError):
            evict.make_select_args(**{**good, **bad}, max_seq_len=40)
    # compaction
    good = dict(key_cache=h(7, 4, 8, 16, 8), value_cache=h(7, 2, 128, 16), block_tables=i(3, 3), kept=i(3, 2, 30), new_seq_lens=i(3))
    a = evict.make_compact_args(**good, scores=f(7, 2, 16))
    assert (a.num_key_heads, a.key_head_size, a.num_value_heads, a.value_head_size) == (4, 64, 2, 128)
    for bad in (dict(key_cache=h(7, 4, 16, 64)), dict(value_cache=h(6, 2, 128, 16)), dict(value_cache=h(7, 2, 128, 16).bfloat16()),
                dict(kept=i(3, 60)), dict(block_tables=i(2, 3)), dict(new_seq_lens=i(4)), dict(key_cache=h(7, 4, 8, 8, 16))):
        with pytest.raises(ValueError):
            evict.make_compact_args(**{**good, **bad})
    with pytest.raises(ValueError):
        evict.make_compact_args(**good, scores=f(7, 2, 15))
    a = evict.make_compact_args(b(7, 2, 576), b(7, 2, 1152), i(3, 3), i(3, 2, 30), i(3), layout="nhd", kv_dtype="e2m1")
    assert (a.key_head_size, a.value_head_size, a.dtype) == (64, 128, _abi.PA_DTYPE_F16)


# ------------------------------------------------------------------ the statements themselves

LEVELS = [Fraction(x) for x in ("0", "0.5", "1", "1.5", "2", "3", "4", "6")]


def _nearest(q, values):
    """Index of the value nearest to q, of two equally near the even one."""
    best = sorted((abs(q - v), i & 1, i) for i, v in enumerate(values))[0]
    return best[2]


def test_quantisation_is_the_nearest_code():
    """Against rational arithmetic, element by element."""
    rng = np.random.default_rng(1)
    scales = [Fraction(float(v)) for v in e4m3_values()[:127]]
    for g in (1.0, 0.0173, 0.0019, 3.0):
        x = (rng.standard_normal((6, 64)) * 2.0 ** rng.integers(-4, 5, (6, 1))).astype(np.float16)
        x[0, :16], x[1, 3] = 0, -0.0
        codes, s = quantise4(x.astype(np.float64), g)
        gf = Fraction(float(np.float32(g)))
        for r in range(6):
            for b in range(4):
                row = [Fraction(float(v)) for v in x[r, 16 * b:16 * b + 16]]
                top = max(abs(v) for v in row)
                c = _nearest(min(top / (6 * gf), Fraction(448)), scales)
                assert c == s[r, b]
                for i, v in enumerate(row):
                    got = codes[r, 8 * b + i // 2] >> (4 * (i & 1)) & 15
                    want = 0 if c == 0 else _nearest(min(abs(v) / (gf * scales[c]), Fraction(6)), LEVELS) | (8 if np.signbit(x[r, 16 * b + i]) else 0)
                    assert got == want, (g, r, b, i)


def test_stored_pages_read_back():
    x = np.random.default_rng(2).standard_normal((20, 2, 64)).astype(np.float16).astype(np.float64)
    c = store4(pages4(3, 2, 64, 0x11), x, np.arange(20) + 5, 0.0019)
    back = values4(c, 0.0019).transpose(0, 2, 1, 3).reshape(48, 2, 64)[5:25]
    top = np.abs(x.reshape(20, 2, 4, 16)).max(-1).repeat(16, -1)
    # half the distance of the two largest codes (1 of 6), of a block scale that is half a step of e4m3 (2^-4) off
    assert np.all(np.abs(back - x) <= top * (1 / 6) * (1 + 2.0 ** -4) + top * 2.0 ** -4)
    untouched = values4(pages4(3, 2, 64, 0x11), 0.0019)
    assert np.array_equal(values4(c, 0.0019).transpose(0, 2, 1, 3).reshape(48, 2, 64)[:5], untouched.transpose(0, 2, 1, 3).reshape(48, 2, 64)[:5])


def test_selection_statement():
    rng = np.random.default_rng(3)
    for _ in range(200):
        n, budget, sink, recent = (int(v) for v in rng.integers(0, 30, 4))
        scores = rng.integers(0, 5, (2, 1, 16)).astype(np.float32)
        scores[rng.random(scores.shape) < 0.1] = np.nan
        kept, new = select_ref(scores, np.array([[1, 0]]), [n], [budget], sink, recent, 30, -1)
        assert new[0] == min(n, budget)
        flat = np.concatenate([scores[1, 0], scores[0, 0]])[:n]
        stay = set(range(n)) if n <= budget else set(range(n - min(recent, budget), n))
        if n > budget:
            stay |= set(range(min(sink, budget - len(stay))))
            rest = sorted((t for t in range(n) if t not in stay), key=lambda t: (np.isnan(flat[t]), -flat[t] if flat[t] == flat[t] else 0, t))
            stay |= set(rest[:budget - len(stay)])
        assert list(kept[0, 0, :new[0]]) == sorted(stay)
        assert np.all(kept[0, 0, new[0]:] == -1)


@pytest.mark.parametrize("layout", ["split", "nhd"])
def test_compaction_statement(layout):
    rng = np.random.default_rng(4)
    ks, vs = ((3, 2, 8, 16, 8), (3, 1, 64, 16)) if layout == "split" else ((3, 2, 16, 64), (3, 1, 16, 64))
    k, v = rng.integers(0, 1000, ks).astype(np.int16), rng.integers(0, 1000, vs).astype(np.int16)
    s = rng.random((3, 1, 16)).astype(np.float32)
    table, kept = np.array([[2, 0, 1]]), np.array([[[0, 3, 18, 40]]])
    nk, nv, ns = compact_ref([k, v], s, table, kept, [4], layout, 1, False)
    for to, src in enumerate(kept[0, 0]):
        a, b, c, d = table[0, to // 16], to % 16, table[0, src // 16], src % 16
        assert ns[a, 0, b] == s[c, 0, d]
        if layout == "nhd":
            assert np.array_equal(nk[a, :, b], k[c, :, d]) and np.array_equal(nv[a, 0, b], v[c, 0, d])
        else:
            assert np.array_equal(nk[a, :, :, b], k[c, :, :, d]) and np.array_equal(nv[a, 0, :, b], v[c, 0, :, d])
    nk[2], nv[2], ns[2] = k[2], v[2], s[2]  # the first page is the only one written
    assert np.array_equal(nk, k) and np.array_equal(nv, v) and np.array_equal(ns, s)
