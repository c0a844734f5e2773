"""GPU tests of pa_diff_decode: every output and partition statistic against the
formula in 64 bits, within the error that diff_ref.py derives."""
from __future__ import annotations

import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import paged_kv_attention_v2_gb300 as pa  # noqa: E402
from diff_ref import diff_ref, make_case  # noqa: E402
from paged_kv_attention_v2_gb300 import _abi  # noqa: E402
from paged_kv_attention_v2_gb300.diff import make_diff_args  # noqa: E402

DEV = "cuda:0"
TYPES = [("f32", None), ("f16", None), ("bf16", None), ("f16", "e4m3"), ("bf16", "e5m2"), ("bf16", "e4m3"), ("f16", "e5m2")]
EDGE = (0, 1, 15, 16, 17, 511, 512, 513, 1100)


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


class Call:
    def __init__(self, c, mode="auto", metadata_ready=False, host_lens=True, **over):
        self.c = c
        rows, heads, _, d = c["query"].shape
        n = len(c["lens"])
        fused = mode == "v2f"
        ws = pa.alloc_diff_workspace(rows, heads, d, c["max_seq_len"], DEV, num_seqs=n if fused else None,
                                     num_kv_heads=c["kv_heads"], tile_counters=mode in ("auto", "v2f"))
        for k in ("exp_sums", "max_logits", "tmp_out"):
            ws[k].fill_(float("nan"))
        self.ws = ws
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.out = torch.full((rows, heads, 2 * d), float("nan"), dtype=c["query"].dtype, device=DEV)
        on = lambda x: None if x is None else x.to(DEV)  # noqa: E731
        self.tensors = [self.out, on(c["query"]), on(c["key_cache"]), on(c["value_cache"]), _int(c["table"]), _int(c["lens"])]
        self.kw = dict(lambdas=on(c["lambdas"]), num_kv_heads=c["kv_heads"], scale=c["scale"], max_seq_len=c["max_seq_len"],
                       norm=c["norm"], norm_weight=on(c["norm_weight"]), norm_eps=c["eps"], out_scale=c["out_scale"],
                       alibi_slopes=on(c["alibi"]), softcap=c["softcap"], layout=c["layout"],
                       mode="v2" if fused else mode, window_left=c["window"], kv_dtype=c["kv"], k_scale=c["k_scale"],
                       v_scale=c["v_scale"], dev_error=self.err, metadata_ready=metadata_ready, **ws)
        if host_lens:
            self.kw["seq_lens_host"] = c["lens"]
        if c["start"] is not None:
            self.kw.update(query_start=_int(c["start"]), max_query_len=int(max(max(c["q_len"]), 1)))
        self.kw.update(over)

    def plan(self):
        return pa.diff_plan(make_diff_args(*self.tensors, **self.kw))

    def run(self, **kw):
        pa.pa_diff_decode(*self.tensors, **self.kw, **kw)
        return self

    def check(self, ref, err=0, what=""):
        torch.cuda.synchronize()
        out, tol, ml, es = ref
        assert int(self.err) == err, (what, int(self.err))
        got = self.out.double().cpu().numpy()
        bad = ~(np.abs(got - out) <= tol)
        if bad.any():
            at = tuple(np.argwhere(bad)[0])
            raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} out of tolerance, first {at}: {got[at]!r} for "
                                 f"{out[at]!r} +- {tol[at]:.3g}; worst {np.nanmax(np.abs(got - out) / np.maximum(tol, 1e-30)):.3g}")
        for name in ("partition_counters", "tile_counters"):
            if self.ws.get(name) is not None:
                assert int(self.ws[name].abs().sum()) == 0, name
        plan = self.plan()
        if plan["mode"] == "v2":  # the statistics of its partitions, at the front of the workspace
            if plan["partition_tokens"] != 512:
                _, _, ml, es = diff_ref(self.c, plan["partition_tokens"])
            for name, want in (("max_logits", ml), ("exp_sums", es)):
                g = self.ws[name].double().cpu().numpy().reshape(-1)[:want.size].reshape(want.shape)
                same = g == want  # unused partitions: exactly -inf and 0
                near = np.abs(np.where(same, 0, g - np.where(np.isinf(want), 0, want))) <= \
                    1e-4 * np.maximum(np.abs(np.where(np.isinf(want), 0, want)), 1)
                assert np.all(same | (near & np.isfinite(want) & ((want != 0) | (name == "max_logits")))), (what, name)
        return got


def _check(c, modes=("v1", "v2", "v2f", "auto"), **kw):
    ref = diff_ref(c)
    for mode in modes:
        call = Call(c, mode, **kw)
        call.run().check(ref, what=mode)
        call.run().check(ref, what=mode + " again")


@pytest.mark.parametrize("layout", ["split", "nhd"])
@pytest.mark.parametrize("size", [64, 128])
@pytest.mark.parametrize("dtype,kv", TYPES)
@pytest.mark.parametrize("kv_heads,group", [(2, 1), (1, 4), (2, 5), (1, 8)])
def test_single_token(dtype, kv, size, layout, kv_heads, group):
    _check(make_case(group, dtype, kv, size, layout, kv_heads, group, EDGE))


@pytest.mark.parametrize("layout", ["split", "nhd"])
@pytest.mark.parametrize("size", [64, 128])
@pytest.mark.parametrize("dtype,kv", TYPES)
@pytest.mark.parametrize("group,most", [(1, 4), (2, 4), (1, 8), (4, 2)])
def test_several_tokens(dtype, kv, size, layout, group, most):
    lens = (2, 16, 17, 512, 514, 1030, 0, 3)
    q_len = [min(1 + i % most, most) for i in range(len(lens))]
    q_len[-1] = most  # more tokens than keys: the first see none
    _check(make_case(most, dtype, kv, size, layout, 2, group, lens, q_len=q_len))


@pytest.mark.parametrize("dtype,kv,size,layout,group", [("f16", None, 64, "split", 4), ("bf16", None, 128, "nhd", 7),
                                                        ("f32", None, 64, "nhd", 3), ("bf16", "e4m3", 64, "nhd", 8),
                                                        ("f16", "e5m2", 128, "split", 2), ("f32", None, 128, "split", 6)])
@pytest.mark.parametrize("opt", [dict(softcap=20.0, mult=2.0), dict(alibi=True), dict(window=0), dict(window=100),
                                 dict(window=600, alibi=True, softcap=30.0), dict(norm=False), dict(weight=False),
                                 dict(per_row=True)], ids=lambda o: "-".join(o))
def test_options(dtype, kv, size, layout, group, opt):
    _check(make_case(5, dtype, kv, size, layout, 2, group, (1, 40, 512, 700, 1537, 0), **opt))
    if group <= 4:
        _check(make_case(6, dtype, kv, size, layout, 1, group, (1, 40, 512, 700, 1537, 0), q_len=[1, 2, 2, 0, 2, 1], **opt))


@pytest.mark.parametrize("dtype,kv,size,layout,group,n,longest", [
    ("bf16", None, 64, "nhd", 7, 2, 40000),      # 79 partitions, few rows: a CTA per row merges
    ("f16", None, 128, "split", 2, 3, 20000),    # 40 partitions
    ("f32", None, 64, "split", 4, 40, 17000),    # 34 partitions of many rows: a warp per map
    ("f16", "e4m3", 128, "nhd", 8, 1, 34000),
    ("f16", "e4m3", 64, "split", 2, 90, 35000),  # 69 partitions of many rows
])
def test_long(dtype, kv, size, layout, group, n, longest):
    lens = np.full(n, 100)
    lens[0], lens[-1] = longest, longest - 777
    _check(make_case(7, dtype, kv, size, layout, 4 if n > 10 else 1, group, lens), modes=("v2", "auto", "v1"))


def test_empty_batch_and_no_rows():
    c = make_case(1, "f16", None, 64, "split", 1, 2, (5, 9))
    call = Call(c)
    call.tensors = [call.out[:0], call.tensors[1][:0], *call.tensors[2:4], call.tensors[4][:0], call.tensors[5][:0]]
    for k in ("exp_sums", "max_logits", "tmp_out"):
        call.kw[k] = call.kw[k][:0]
    call.kw["seq_lens_host"] = c["lens"][:0]
    call.run()
    torch.cuda.synchronize()
    assert torch.isnan(call.out).all()


@pytest.mark.parametrize("mode", ["v1", "v2"])
def test_masked_rows_of_a_padded_batch_stay(mode):
    """Rows behind the last token (a padded batch) are left as they were."""
    c = make_case(2, "bf16", None, 64, "split", 2, 2, (30, 600), q_len=[2, 1])
    call = Call(c, mode)
    big = torch.full((7,) + tuple(call.out.shape[1:]), 7.0, dtype=call.out.dtype, device=DEV)
    call.tensors[0] = call.out = big[:3]
    call.run().check(diff_ref(c))
    assert (big[3:] == 7).all()


@pytest.mark.parametrize("mode", ["v1", "v2", "v2f", "auto"])
@pytest.mark.parametrize("q_len", [[2, 1, 0], [0, 0, 0]])
def test_rows_behind_the_last_token_of_the_call_stay(mode, q_len):
    """A call padded to eight rows, in the workspace of a larger batch still."""
    c = make_case(5, "bf16", "e4m3", 64, "nhd", 2, 2, (30, 1600, 0), q_len=[2, 1, 0], per_row=True)
    call = Call(c, mode)
    wide = lambda t, v: torch.cat([t, torch.full((8 - t.shape[0],) + tuple(t.shape[1:]), v, dtype=t.dtype, device=DEV)])  # noqa: E731
    nan = float("nan")
    call.tensors[0] = out = wide(call.tensors[0], 7.0)
    call.tensors[1] = wide(call.tensors[1], nan)
    call.kw["lambdas"] = wide(call.kw["lambdas"], nan)
    call.kw["query_start"] = _int(np.concatenate([[0], np.cumsum(q_len)]))
    room = pa.alloc_diff_workspace(11, 4, 64, 5000, DEV, num_seqs=9 if mode == "v2f" else None, num_kv_heads=3)
    call.kw.update(room)
    call.ws.update(room)
    rows = sum(q_len)
    if rows == 0:
        out.fill_(7.0)
    for _ in range(2):
        call.run()
    torch.cuda.synchronize()
    assert (out[rows:] == 7).all()
    if rows:
        call.out = out[:rows]
        call.check(diff_ref(c))
    assert int(call.err) == 0


def test_no_rows_of_several_sequences():
    c = make_case(6, "f16", None, 64, "split", 2, 2, (30, 600), q_len=[1, 1])
    call = Call(c, "v2")
    call.tensors[0], call.tensors[1] = call.tensors[0][:0].clone(), call.tensors[1][:0].clone()
    call.kw["query_start"] = _int([0, 0, 0])
    call.run()
    torch.cuda.synchronize()
    assert int(call.err) == 0


@pytest.mark.parametrize("mode", ["v1", "v2", "v2f"])
def test_bad_metadata_is_reported_and_harmless(mode):
    c = make_case(3, "f16", None, 64, "nhd", 2, 3, (100, 600, 40))
    call = Call(c, mode)
    call.tensors[4][1, 3] = 10 ** 6
    call.tensors[4][1, 20] = -5
    call.run()
    torch.cuda.synchronize()
    assert int(call.err) == pa.PA_DEVERR_BLOCK_ID
    good = diff_ref(c)
    got = call.out.double().cpu().numpy()
    assert np.all(np.abs(got - good[0])[[0, 2]] <= good[1][[0, 2]])
    call = Call(c, mode)
    call.tensors[5][0] = -3
    call.tensors[5][2] = 601
    call.run()
    torch.cuda.synchronize()
    assert int(call.err) & pa.PA_DEVERR_SEQ_LEN
    assert (call.out[0] == 0).all()


@pytest.mark.parametrize("dtype,kv,mode", [("f16", None, "v2"), ("bf16", "e4m3", "v1"), ("f32", None, "v2")])
@pytest.mark.parametrize("size", [64, 128])
def test_withheld_page_times_out_and_context_survives(dtype, kv, mode, size):
    c = make_case(4, dtype, kv, size, "split", 2, 5, (700, 1300, 90))
    ref = diff_ref(c)
    lib = _abi.load()
    assert lib.pa_debug_withhold_page(1, 50_000_000) == 0
    try:
        t0 = time.perf_counter()
        call = Call(c, mode).run()
        torch.cuda.synchronize()
        assert int(call.err) & pa.PA_DEVERR_TIMEOUT and time.perf_counter() - t0 < 30
    finally:
        assert lib.pa_debug_withhold_page(0, 0) == 0
    Call(c, mode).run().check(ref)


def test_plans():
    """Few tiles merge in the partition kernel, short batches take one pass, unequal ones the dynamic schedule."""
    c = make_case(8, "f16", None, 64, "split", 2, 3, (700, 1300))
    assert Call(c, "v2f").plan()["merge_in_kernel"] and Call(c, "v2f").plan()["kernels"] == 1
    assert Call(c, "v2").plan()["kernels"] == 2
    assert Call(c, "auto").plan()["dynamic_schedule"]
    assert Call(make_case(8, "f16", None, 64, "split", 2, 3, (70, 500))).plan()["mode"] == "v1"


@pytest.mark.parametrize("mode", ["v1", "v2", "v2f", "auto"])
def test_back_to_back_with_metadata_ready_graph_and_stream(mode):
    c = make_case(9, "bf16", None, 64, "nhd", 2, 4, (700, 1300, 5, 2000), q_len=[2, 1, 2, 2])
    ref = diff_ref(c)
    call = Call(c, mode, metadata_ready=True)
    for _ in range(3):
        call.run()
    call.check(ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call.out.fill_(float("nan"))
    side.wait_stream(torch.cuda.current_stream())
    call.run(stream=side)
    call.check(ref)
    call = Call(c, mode)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call.run()
        call.run()
    for _ in range(2):
        call.out.fill_(float("nan"))
        g.replay()
        call.check(ref)


@pytest.mark.parametrize("layout", ["split", "nhd"])
@pytest.mark.parametrize("dtype,kv", [("f16", None), ("bf16", "e4m3")])
def test_pages_past_32_bits(dtype, kv, layout):
    """The last pages of caches of 2.3e9 elements."""
    c = make_case(10, dtype, kv, 64, layout, 8, 1, (70, 600), spare=8)
    small = c["key_cache"].shape[0]
    blocks = 140000
    call = Call(c, "v2")
    for i in (2, 3):
        page = call.tensors[i]
        big = torch.zeros((blocks,) + tuple(page.shape[1:]), dtype=torch.uint8 if kv else page.dtype, device=DEV)
        big[blocks - small:] = page.view(big.dtype)
        call.tensors[i] = big
    call.tensors[4] += blocks - small
    call.run().check(diff_ref(c))


def test_identical_maps_cancel_and_lambda_zero_is_plain_attention():
    """With both maps the same and lambda one nothing is left; with lambda zero,
    no norm and out_scale one, it is pa_decode of the first map's keys."""
    c = make_case(11, "f16", None, 64, "nhd", 2, 2, (600, 33), norm=False)
    c["query"][:, :, 1] = c["query"][:, :, 0]
    c["key_cache"][:, 1::2] = c["key_cache"][:, 0::2]
    c["lambdas"].fill_(1.0)
    c["out_scale"] = 1.0
    for mode in ("v1", "v2", "v2f"):
        assert (Call(c, mode).run().out == 0).all()
    c = make_case(12, "f16", None, 64, "nhd", 2, 2, (600, 33), norm=False)
    c["lambdas"].zero_()
    c["out_scale"] = 1.0
    a = Call(c, "v2").run()
    half = []
    for part in (slice(0, 64), slice(64, 128)):
        out = torch.empty((2, 4, 64), dtype=torch.float16, device=DEV)
        pa.pa_decode(out, a.tensors[1][:, :, 0].contiguous(), a.tensors[2][:, 0::2].contiguous(),
                     a.tensors[3][..., part].contiguous(), a.tensors[4], a.tensors[5], num_kv_heads=2, scale=c["scale"],
                     max_seq_len=c["max_seq_len"], layout="nhd", mode="v2",
                     **pa.alloc_workspace(2, 4, 64, c["max_seq_len"], DEV))
        half.append(out)
    # both are within half a step of fp16 P (2^-11) and of the output of the same sums
    ref = diff_ref(c)
    assert np.all(np.abs((a.out - torch.cat(half, 2)).double().cpu().numpy()) <= 2 * ref[1])


@pytest.mark.parametrize("n,longest,kv_heads,group,low,high", [
    (128, 1200, 4, 2, 1, 4),       # a warp merges both maps
    (24, 6000, 2, 4, 5, 32),       # two warps per row
    (1, 30000, 2, 2, 33, 64),      # few rows of many partitions: a CTA per row
    (3, 34000, 1, 5, 65, 100),
])
def test_every_merge(n, longest, kv_heads, group, low, high):
    """Each kernel that merges partitions, by the number of them the plan shows."""
    c = make_case(13, "bf16", None, 64, "nhd", kv_heads, group, np.full(n, longest), alibi=True)
    call = Call(c, "v2")
    tokens = call.plan()["partition_tokens"]
    assert low <= -(-longest // tokens) <= high and tokens % 16 == 0, tokens
    call.run().check(diff_ref(c))


@pytest.mark.parametrize("dtype,kv,size,group", [("f32", None, 64, 4), ("f32", None, 64, 7), ("f32", None, 128, 2),
                                                 ("f16", None, 64, 8), ("bf16", None, 128, 3), ("f16", "e4m3", 64, 8)])
def test_calls_repeat_bit_for_bit(dtype, kv, size, group):
    """Short sequences, whose page tails are zeroed, beside long ones: a stage handed
    back before its last read has returned shows as calls that differ."""
    lens = np.full(40, 97)
    lens[0], lens[-1] = 17000, 16223
    c = make_case(14, dtype, kv, size, "split", 4, group, lens)
    call = Call(c, "v2", host_lens=False)
    first, differ = call.run().out.clone(), torch.zeros((), device=DEV)
    for _ in range(400):
        differ += (call.run().out != first).any()
    assert int(differ) == 0 and not torch.isnan(first).any()


@pytest.mark.parametrize("layout", ["split", "nhd"])
@pytest.mark.parametrize("size,group", [(64, 3), (64, 8), (128, 1), (128, 7)])
def test_identical_maps_cancel_in_fp32(layout, size, group):
    """Both maps take the same sums in the same order, whichever lanes or warps hold them."""
    c = make_case(14, "f32", None, size, layout, 2, group, (1600, 33, 0, 250), norm=False, softcap=20.0, alibi=True)
    c["query"][:, :, 1] = c["query"][:, :, 0]
    c["key_cache"][:, 1::2] = c["key_cache"][:, 0::2]
    c["lambdas"].fill_(1.0)
    for mode in ("v1", "v2", "v2f"):
        assert (Call(c, mode).run().out == 0).all()
