"""Host-side checks of pa_diff_decode (no GPU): the struct matches the header and
refusals come before anything is launched; the 64-bit statement the GPU tests
compare with is itself compared with a plain loop."""
import ctypes
import math
import pathlib
import shutil
import subprocess

import numpy as np
import pytest

import paged_kv_attention_v2_gb300 as pa
from diff_ref import diff_ref, make_case
from paged_kv_attention_v2_gb300 import _abi
from paged_kv_attention_v2_gb300.diff import make_diff_args

torch = pytest.importorskip("torch")
INC = pathlib.Path(__file__).resolve().parents[1] / "include"


@pytest.fixture(scope="module")
def lib():
    from paged_kv_attention_v2_gb300 import build
    build.build()
    return _abi.load()


def test_struct_layout_matches_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines = ['#include <stdio.h>', '#include "pa_decode.h"', "int main(void) {",
             'printf("size %zu\\n", sizeof(pa_diff_args));']
    lines += [f'printf("{f} %zu\\n", offsetof(pa_diff_args, {f}));' for f, _ in _abi.PaDiffArgs._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0;", "}"]) + "\n")
    subprocess.run([cc, "-std=c11", "-I", str(INC), str(src), "-o", str(tmp_path / "layout")], check=True)
    out = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout
    got = {line.split()[0]: int(line.split()[1]) for line in out.splitlines()}
    assert got["size"] == ctypes.sizeof(_abi.PaDiffArgs)
    for f, _ in _abi.PaDiffArgs._fields_:
        assert got[f] == getattr(_abi.PaDiffArgs, f).offset, f


def _args(**over):
    d = _abi.PaDecodeArgs(
        out=16, query=16, key_cache=16, value_cache=16, block_tables=16, seq_lens=16, num_seqs=2, num_heads=8,
        num_kv_heads=2, head_size=64, num_blocks=10, block_size=16, max_seq_len=100, max_blocks_per_seq=7, scale=0.1,
        dtype=_abi.PA_DTYPE_F16, layout=_abi.PA_LAYOUT_SPLIT, mode=_abi.PA_MODE_V2, exp_sums=16, max_logits=16, tmp_out=16)
    a = _abi.PaDiffArgs(d, 16, 0, None, 1e-5, 1.0, 1)
    for k, v in over.items():
        setattr(a if hasattr(a, k) else a.decode, k, v)
    return a


@pytest.mark.parametrize("over,expect", [
    ({"num_heads": 18}, _abi.PA_ERR_UNSUPPORTED),                # group 9: 18 columns
    ({"num_heads": 7}, _abi.PA_ERR_INVALID_ARG),
    ({"head_size": 32}, _abi.PA_ERR_UNSUPPORTED),
    ({"head_size": 256}, _abi.PA_ERR_UNSUPPORTED),
    ({"block_size": 32}, _abi.PA_ERR_UNSUPPORTED),
    ({"lambdas": None}, _abi.PA_ERR_INVALID_ARG),
    ({"lambdas": 18}, _abi.PA_ERR_INVALID_ARG),
    ({"norm_weight": 2}, _abi.PA_ERR_INVALID_ARG),
    ({"lambda_row_stride": -1}, _abi.PA_ERR_INVALID_ARG),
    ({"norm_eps": 0.0}, _abi.PA_ERR_INVALID_ARG),
    ({"norm_eps": float("nan")}, _abi.PA_ERR_INVALID_ARG),
    ({"out_scale": float("inf")}, _abi.PA_ERR_INVALID_ARG),
    ({"tmp_out": None}, _abi.PA_ERR_WORKSPACE),
    ({"query": None}, _abi.PA_ERR_INVALID_ARG),
    ({"max_seq_len": (1 << 30) + 1, "max_blocks_per_seq": 1 << 27}, _abi.PA_ERR_UNSUPPORTED),
    ({"out": 8}, _abi.PA_ERR_INVALID_ARG),
    ({"kv_dtype": _abi.PA_KV_FP8_E4M3, "dtype": _abi.PA_DTYPE_F32}, _abi.PA_ERR_UNSUPPORTED),
    ({"query_start": 16, "num_query_tokens": 4, "max_query_len": 3}, _abi.PA_ERR_UNSUPPORTED),  # 4 heads x 3 > 8
    ({"query_start": 16, "num_query_tokens": 4, "max_query_len": 0}, _abi.PA_ERR_INVALID_ARG),
    ({"num_seqs": 0}, _abi.PA_OK),
    ({"query_start": 16, "num_query_tokens": 0, "max_query_len": 1, "query": None, "out": None}, _abi.PA_OK),
])
def test_refusals(lib, over, expect):
    assert lib.pa_diff_decode(ctypes.byref(_args(**over)), None) == expect
    plan = _abi.PaLaunchPlan()
    assert lib.pa_diff_plan(ctypes.byref(_args(**over)), ctypes.byref(plan)) == expect


def test_null(lib):
    assert lib.pa_diff_decode(None, None) == _abi.PA_ERR_INVALID_ARG
    assert lib.pa_diff_plan(None, ctypes.byref(_abi.PaLaunchPlan())) == _abi.PA_ERR_INVALID_ARG
    assert lib.pa_diff_plan(ctypes.byref(_args()), None) == _abi.PA_ERR_INVALID_ARG


def test_binding_refuses_what_only_the_tensors_know():
    c = make_case(1, "f16", None, 64, "split", 2, 2, (20, 40))
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32))  # noqa: E731
    out = torch.empty((2, 4, 128), dtype=torch.float16)
    good = dict(out=out, query=c["query"], key_cache=c["key_cache"], value_cache=c["value_cache"],
                block_tables=i32(c["table"]), seq_lens=i32(c["lens"]))
    kw = dict(lambdas=c["lambdas"], num_kv_heads=2, scale=0.1, max_seq_len=40)
    make_diff_args(**good, **kw)
    make_diff_args(**good, **{**kw, "lambdas": torch.zeros(2, 4)})
    with pytest.raises(ValueError):
        pa.pa_diff_decode(*good.values(), **kw)                      # not on a GPU
    for bad in (dict(query=c["query"][:, :, 0]), dict(out=out[:, :, :64]), dict(out=out.float()),
                dict(query=c["query"][:1], out=out[:1]), dict(key_cache=c["key_cache"][:, :2].contiguous()),
                dict(value_cache=c["value_cache"][:-1]), dict(value_cache=c["value_cache"].view(torch.bfloat16)), dict(value_cache=c["value_cache"].float()),
                dict(key_cache=c["key_cache"].transpose(0, 1)), dict(block_tables=i32(c["table"]).long()),
                dict(block_tables=i32(c["table"][:1]))):
        with pytest.raises(ValueError):
            make_diff_args(**{**good, **bad}, **kw)
    for bad in (dict(lambdas=torch.zeros(3)), dict(lambdas=torch.zeros(4, dtype=torch.float64)),
                dict(lambdas=torch.zeros(1, 4)), dict(norm_weight=torch.zeros(64)), dict(kv_dtype="e4m3"),
                dict(query_start=i32([0, 1, 2])), dict(exp_sums=torch.zeros(3)), dict(tile_counters=i32([0])),
                dict(seq_lens_host=np.zeros(3))):
        with pytest.raises(ValueError):
            make_diff_args(**good, **{**kw, **bad})


def test_statement_in_64_bits_against_a_loop():
    c = make_case(2, "f32", None, 64, "split", 2, 2, (5, 19), q_len=[2, 1], softcap=3.0, alibi=True, window=6, per_row=True)
    out, tol, ml, es = diff_ref(c)
    k = c["key_cache"].permute(0, 3, 1, 2, 4).flatten(3).double()  # [block, offset, head, d]
    v = c["value_cache"].permute(0, 3, 1, 2).double()
    for s, (r0, n) in enumerate(((0, 2), (2, 1))):
        for i in range(n):
            pos = int(c["lens"][s]) - n + i
            for h in range(4):
                maps = []
                for m in (0, 1):
                    z, rows = [], []
                    for t in range(max(0, pos - 6), pos + 1):
                        b, o = c["table"][s][t // 16], t % 16
                        x = float(np.float32(c["scale"])) * sum(float(a) * float(b_) for a, b_ in
                                                                zip(c["query"][r0 + i, h, m], k[b, o, 2 * (h // 2) + m]))
                        z.append(3.0 * math.tanh(x / 3.0) + float(c["alibi"][h]) * t)
                        rows.append(v[b, o, h // 2])
                    p = [math.exp(x - max(z)) for x in z]
                    maps.append(sum(w / sum(p) * row for w, row in zip(p, rows)))
                    assert abs(ml[r0 + i, h, m, 0] - max(z)) < 1e-12 and abs(es[r0 + i, h, m, 0] - sum(p)) < 1e-12
                x = maps[0] - float(c["lambdas"][r0 + i, h]) * maps[1]
                y = 0.4 * c["norm_weight"].double() * x / torch.sqrt((x * x).mean() + 1e-5)
                assert np.allclose(out[r0 + i, h], y.numpy(), rtol=1e-12, atol=1e-12)
    assert np.isfinite(tol).all() and (tol > 0).all()


@pytest.mark.parametrize("cls", [_abi.PaDiffArgs, _abi.PaTablesArgs, _abi.PaAppendArgs])
def test_packed_arguments_are_the_struct(cls):
    """The packed bytes have the struct's size and every field in its place."""
    def leaves(c, base=0):
        for name, t in c._fields_:
            at = base + getattr(c, name).offset
            if issubclass(t, ctypes.Structure):
                yield from leaves(t, at)
            else:
                yield at, t
    fields = list(leaves(cls))
    pack = _abi.packer(cls)
    assert pack.size == ctypes.sizeof(cls)
    data = pack.pack(*range(1, len(fields) + 1))
    for i, (at, t) in enumerate(fields):
        assert t.from_buffer_copy(data, at).value == i + 1


def test_binding_takes_the_workspace_of_a_larger_batch():
    c = make_case(1, "f16", None, 64, "split", 2, 2, (20, 40))
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32))  # noqa: E731
    args = (torch.empty((2, 4, 128), dtype=torch.float16), c["query"], c["key_cache"], c["value_cache"], i32(c["table"]),
            i32(c["lens"]))
    kw = dict(lambdas=c["lambdas"], num_kv_heads=2, scale=0.1, max_seq_len=40)
    room = dict(exp_sums=torch.empty(5, 4, 2, 3), max_logits=torch.empty(5, 4, 2, 3), tmp_out=torch.empty(5, 4, 2, 3, 128),
                partition_counters=torch.zeros((5, 2), dtype=torch.int32))
    make_diff_args(*args, **kw, **room)
    for name, t in room.items():  # one element less than this call needs
        need = {"exp_sums": 16, "max_logits": 16, "tmp_out": 16 * 128, "partition_counters": 4}[name]
        make_diff_args(*args, **kw, **{name: t.flatten()[:need]})
        with pytest.raises(ValueError):
            make_diff_args(*args, **kw, **{name: t.flatten()[:need - 1]})
