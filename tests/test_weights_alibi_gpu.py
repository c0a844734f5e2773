"""GPU tests of pa_add_weights after a pa_decode with ALiBi over long sequences, where a maximum at an
absolute position (slope x position) has few bits left: relative_max keeps them.  Weights against the
softmax in 64 bits."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import paged_kv_attention_v2_gb300 as pa  # noqa: E402
from short_ref import pages4, store4, values4  # noqa: E402

DEV = "cuda:0"
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
# As without ALiBi (test_evict_gpu): a logit's terms add up to about 7, and 1e-4 is over a hundred half steps of
# fp32 of that; twice, in the level and in the logit.  ALiBi adds slope x distance, rounded relative to the last
# token: tokens with a weight of 1e-30 and more are within 80 of the maximum, half a step of fp32 there 4e-6, once
# in the logit, and up to four times (two in the tile, two between tiles) in the level.
REL = 2e-4


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _cache(rng, gen, kv, dtype, layout, blocks, kv_heads, size):
    """(cache on the GPU as stored, what it stands for [blocks, kv heads, 16, size] in 64 bits, k_scale)."""
    rows = torch.randn((blocks, kv_heads, 16, size), generator=gen)
    if kv == "e2m1":
        flat = rows.half().double().numpy().transpose(0, 2, 1, 3).reshape(-1, kv_heads, size)
        c = store4(pages4(blocks, kv_heads, size), flat, np.arange(blocks * 16), 0.0019)
        return torch.from_numpy(c).to(DEV), torch.from_numpy(values4(c, 0.0019)).to(DEV), 0.0019
    ks = 2.0 ** -5 if kv else 1.0
    c = (rows / ks).to(FP8[kv] if kv else TORCH[dtype])
    values = c.double().to(DEV) * ks
    if layout == "split":
        x = 16 // c.element_size()
        c = c.unflatten(3, (size // x, x)).permute(0, 1, 3, 2, 4)
    return c.contiguous().to(DEV), values, ks


def _run(dtype, kv, layout, size, kv_heads, lens, slopes, q_len=None, window=-1, cap=0.0, fused=False, graph=False,
         relative=True, seed=0):
    """(scores, weights in 64 bits, the workspace), scores of zero before the call."""
    rng, gen = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    n, heads = len(lens), len(slopes)
    group = heads // kv_heads
    own = [-(-x // 16) for x in lens]
    ids = rng.permutation(sum(own))
    table = np.zeros((n, max(own)), dtype=np.int64)
    at = np.concatenate([[0], np.cumsum(own)])
    for s in range(n):
        table[s, :own[s]] = ids[at[s]:at[s + 1]]
    cache, values, ks = _cache(rng, gen, kv, dtype, layout, len(ids), kv_heads, size)
    start = np.concatenate([[0], np.cumsum(q_len)]) if q_len else np.arange(n + 1)
    rows, top, scale = int(start[-1]), max(lens), size ** -0.5
    q = torch.randn((rows, heads, size), generator=gen).to(TORCH[dtype]).to(DEV)
    slope = torch.tensor(slopes, dtype=torch.float32, device=DEV)
    err = _int([0])
    kw = dict(num_kv_heads=kv_heads, scale=scale, max_seq_len=top, layout=layout, kv_dtype=kv, k_scale=ks, window_left=window,
              softcap=cap, alibi_slopes=slope, dev_error=err, relative_max=relative)
    if q_len:
        kw.update(query_start=_int(start), max_query_len=max(q_len))
    ws = pa.alloc_workspace(n, heads, size, top, DEV, num_query_tokens=rows if q_len else None,
                            num_kv_heads=kv_heads if fused else None)
    raw = cache.view(torch.uint8) if kv else cache
    vc = raw if layout == "nhd" else raw.reshape(len(ids), kv_heads, size, 16)
    scores = torch.zeros((len(ids), kv_heads, 16), device=DEV)
    tg, lg, out = _int(table), _int(lens), torch.empty_like(q)

    def step():
        pa.pa_decode(out, q, raw, vc, tg, lg, mode="v2", **kw, **ws)
        pa.pa_add_weights(scores, q, cache, tg, lg, ws["exp_sums"], ws["max_logits"], decay=0.0, **kw)
    step()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        scores.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert int(err) == 0
    want = torch.zeros((len(ids), kv_heads, 16), dtype=torch.float64, device=DEV)
    for s, length in enumerate(lens):
        t = torch.arange(length, device=DEV)
        blk = tg[s].long()[t // 16]
        k = values[blk, :, t % 16]                                                  # [t, kv heads, size]
        added = torch.zeros((length, kv_heads), dtype=torch.float64, device=DEV)
        for r in range(start[s], start[s + 1]):
            pos = length - (int(start[s + 1]) - r)
            z = torch.einsum("hgd,thd->hgt", q[r].double().view(kv_heads, group, size), k) * scale
            z = cap * torch.tanh(z / cap) if cap > 0 else z
            z = z + slope.double().view(kv_heads, group, 1) * t
            seen = (t <= pos) & ((t >= pos - window) if window >= 0 else True)
            added += torch.softmax(z.masked_fill(~seen, -math.inf), -1).sum(1).t()
        want[blk, :, t % 16] = added
    return scores.double(), want, ws, (q, values, tg, slope, out)


def _worst(got, want):
    """Largest error of a weight above 1e-30 relative to itself."""
    return float(((got - want).abs() / want.clamp(min=1e-30)).masked_fill(want < 1e-30, 0).max())


STEEP = [0.9, 0.82, 0.5, 0.31, 0.11, 0.0625, 0.0173, 0.004]
KINDS = [("f16", None, "split"), ("bf16", None, "nhd"), ("f32", None, "nhd"), ("f16", "e4m3", "split"), ("bf16", "e5m2", "nhd"),
         ("bf16", "e2m1", "nhd"), ("f16", "e2m1", "nhd")]


@pytest.mark.parametrize("dtype,kv,layout", KINDS)
def test_long_sequences(dtype, kv, layout):
    got, want, _, _ = _run(dtype, kv, layout, 64, 2, [30011, 100003], STEEP, graph=True)
    assert _worst(got, want) <= REL
    assert bool((got[want < 1e-30] < 2e-30).all())


@pytest.mark.parametrize("dtype,kv,layout", KINDS)
def test_every_merge(dtype, kv, layout):
    """In the partition kernel, a warp to each row (the statistics of many rows), a CTA to each row."""
    for lens, fused in (([3900, 2000], True), ([1, 17, 16000] + [700] * 30, False), ([70001], False)):
        got, want, _, _ = _run(dtype, kv, layout, 64, 2, lens, STEEP, fused=fused)
        assert _worst(got, want) <= REL, lens


def test_several_tokens_windows_and_softcap():
    for kw in (dict(q_len=[4, 1, 3]), dict(q_len=[2, 4, 1], window=900), dict(cap=20.0), dict(window=5000)):
        for dtype, kv, layout in (("f16", None, "split"), ("bf16", "e2m1", "nhd")):
            got, want, _, _ = _run(dtype, kv, layout, 128, 1, [40, 33000, 20001], [0.9, 0.3, 0.05, 0.01], **kw)
            assert _worst(got, want) <= REL, (kw, dtype)


@pytest.mark.parametrize("lens,fused", [([60001], False), ([3000, 800], True), ([9000] * 40, False)])
def test_relative_statistics_are_the_absolute_ones_without_the_shift(lens, fused):
    """Everything else a decode leaves is the same, bit for bit."""
    a = _run("f16", None, "split", 64, 2, lens, STEEP, fused=fused, relative=False)
    b = _run("f16", None, "split", 64, 2, lens, STEEP, fused=fused)
    assert torch.equal(a[3][4], b[3][4]) and torch.equal(a[2]["exp_sums"], b[2]["exp_sums"])
    ma, mb = a[2]["max_logits"].double(), b[2]["max_logits"].double()
    shift = torch.tensor(STEEP, dtype=torch.float32, device=DEV).double()[None, :, None] * \
        (torch.tensor(lens, device=DEV) - 1).double()[:, None, None]
    there = torch.isfinite(mb)
    assert torch.equal(there, torch.isfinite(ma)) and bool((mb[~there] == -math.inf).all())
    # two roundings of numbers of up to the shift, plus a few of the maxima themselves (below 8)
    assert bool(((ma - mb - shift).abs() <= 2.0 ** -23 * (shift + mb.abs() + 8))[there].all())


def test_absolute_statistics_are_as_far_off_as_stated():
    """Without relative_max: 2^-23 x slope x length on all weights of a row."""
    for length in (2000, 30011):
        got, want, _, _ = _run("f16", None, "split", 64, 2, [length], STEEP, relative=False)
        assert _worst(got, want) <= REL + 2.0 ** -23 * STEEP[0] * length * 1.01


def test_without_slopes_the_flag_changes_nothing():
    a = _run("bf16", "e2m1", "nhd", 64, 1, [5000, 40], [0.0] * 4, relative=False)
    b = _run("bf16", "e2m1", "nhd", 64, 1, [5000, 40], [0.0] * 4)
    assert torch.equal(a[0], b[0]) and torch.equal(a[2]["max_logits"], b[2]["max_logits"])


@pytest.mark.parametrize("n,tokens,counters", [(3, 40001, False), (2, 3000, True), (40, 1500, False)])
def test_differential_statistics_follow_the_flag(n, tokens, counters):
    """pa_diff_decode leaves its statistics by the same field: the outputs and sums are the same, the maxima those
    without the shift."""
    from paged_kv_attention_v2_gb300 import _abi, diff
    gen = torch.Generator().manual_seed(tokens)
    heads, size, pages = 4, 64, -(-tokens // 16)
    q = torch.randn((n, heads, 2, size), generator=gen).half().to(DEV)
    k = torch.randn((pages, 2 * heads, 16, size), generator=gen).half().to(DEV)
    v = torch.randn((pages, heads, 16, 2 * size), generator=gen).half().to(DEV)
    table, lens = _int(np.tile(np.arange(pages), (n, 1))), _int([tokens] * n)
    slope, lam = torch.tensor(STEEP[:heads], device=DEV), torch.rand(heads, generator=gen).to(DEV)
    results = []
    for flag in (0, 1):
        ws = pa.alloc_diff_workspace(n, heads, size, tokens, DEV, num_seqs=n if counters else None, num_kv_heads=heads if counters else None)
        out, err = torch.empty((n, heads, 2 * size), dtype=q.dtype, device=DEV), _int([0])
        a = diff.make_diff_args(out, q, k, v, table, lens, lambdas=lam, num_kv_heads=heads, scale=size ** -0.5, max_seq_len=tokens,
                                alibi_slopes=slope, layout="nhd", mode="v2", dev_error=err, **ws)
        a.decode.relative_max = flag
        plan = diff.diff_plan(a)
        assert _abi.load().pa_diff_decode(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == _abi.PA_OK
        torch.cuda.synchronize()
        assert int(err) == 0 and plan["mode"] == "v2"
        parts = -(-tokens // plan["partition_tokens"])
        results.append((out, *(ws[x].flatten()[:n * heads * 2 * parts].view(n, heads, 2, parts) for x in ("exp_sums", "max_logits"))))
    (oa, ea, ma), (ob, eb, mb) = results
    assert torch.equal(oa, ob) and torch.equal(ea, eb) and bool(torch.isfinite(mb).all())
    shift = slope.double()[None, :, None, None] * (tokens - 1)
    assert bool(((ma.double() - mb.double() - shift).abs() <= 2.0 ** -23 * (shift + mb.double().abs() + 8)).all())
