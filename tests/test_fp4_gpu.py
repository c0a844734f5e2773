"""GPU tests of 4-bit caches: pa_append_kv bit for bit against the definition in 64 bits
(special values, scales whose quotients end next to the border of two codes), and
pa_decode over such pages against the formula in 64 bits."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import paged_kv_attention_v2_gb300 as pa  # noqa: E402
from short_ref import attention, pages4, sequences, store4, values4  # noqa: E402

DEV = "cuda:0"
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}
# half a step of the output, plus half a step of 16 bits of the weights of values up to 5,
# and what 2e-5 of the logits' sums makes of those
TOL = {"f16": (6e-3, 2.0 ** -11), "bf16": (6e-3, 2.0 ** -8)}


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _append(key, value, slots, blocks, ks=1.0, vs=1.0, byte=0x5a):
    """(caches after the call, caches by the definition) of rows on the GPU."""
    caches, want = [], []
    for x, g in ((key, ks), (value, vs)):
        c = pages4(blocks, x.shape[1], x.shape[2], byte)
        caches.append(torch.from_numpy(c).to(DEV))
        want.append(store4(c, x.double().cpu().numpy(), slots, g))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_append_kv(key, value, *caches, _int(slots), layout="nhd", kv_dtype="e2m1", k_scale=ks, v_scale=vs, dev_error=err)
    return [c.cpu().numpy() for c in caches], want, int(err)


def _same(got, want):
    for g, w in zip(got, want):
        assert np.array_equal(g, w), np.argwhere(g != w)[:4]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tokens,k_heads,k_size,v_heads,v_size", [
    (1, 1, 64, 1, 64), (3, 2, 128, 2, 128), (40, 4, 64, 2, 128), (33, 3, 128, 5, 64), (777, 2, 128, 2, 128), (5000, 8, 128, 8, 128)])
def test_append_is_the_definition(tokens, k_heads, k_size, v_heads, v_size, dtype):
    rng, gen = np.random.default_rng(tokens), torch.Generator().manual_seed(tokens)
    blocks = -(-tokens // 16) + 5
    slots = rng.permutation(blocks * 16)[:tokens]
    if tokens > 16:  # successive places from inside a page on, and padding
        slots = np.arange(tokens) + 7
        slots[-3:] = -1
    mag = lambda *s: torch.exp2(torch.randint(-6, 7, s + (1,), generator=gen).float())  # noqa: E731
    key = (torch.randn((tokens, k_heads, k_size), generator=gen) * mag(tokens, k_heads)).to(TORCH[dtype]).to(DEV)
    value = (torch.randn((tokens, v_heads, v_size), generator=gen) * mag(tokens, v_heads)).to(TORCH[dtype]).to(DEV)
    for ks, vs in ((1.0, 0.0019), (0.0173, 2.0 ** -9), (3.3, 1.5)):
        got, want, err = _append(key, value, slots, blocks, ks, vs)
        _same(got, want)
        assert err == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append_rows_of_a_fused_projection(dtype):
    gen = torch.Generator().manual_seed(5)
    row = torch.randn((50, 4 * 64 + 2 * 64 + 2 * 128), generator=gen).to(TORCH[dtype]).to(DEV)
    key, value = row[:, 256:384].unflatten(1, (2, 64)), row[:, 384:].unflatten(1, (2, 128))
    slots = np.random.default_rng(5).permutation(96)[:50]
    got, want, err = _append(key, value, slots, 6)
    _same(got, want)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append_special_values(dtype):
    """NaN, infinities, zeros of both signs, subnormals, the largest numbers, a scale of zero."""
    t = TORCH[dtype]
    top, tiny = torch.finfo(t).max, torch.finfo(t).smallest_normal / 16
    odd = [float("nan"), float("inf"), -float("inf"), 0.0, -0.0, top, -top, tiny, -tiny, 1.0, -1.0]
    gen = torch.Generator().manual_seed(9)
    x = torch.randn((64, 2, 64), generator=gen).to(t)
    pick = torch.randint(0, len(odd), x.shape, generator=gen)
    some = torch.rand((64, 2, 4, 1), generator=gen).expand(64, 2, 4, 16).reshape(x.shape)  # none, few or all of a block
    x = torch.where(torch.rand(x.shape, generator=gen) < some - 0.4, torch.tensor(odd).to(t)[pick], x)
    x[0], x[1], x[2], x[3] = 0.0, -0.0, tiny, top
    x = x.to(DEV)
    for g in (1.0, 0.0173, 2.0 ** -100, 2.0 ** 100, 1e-36, 1e36, 3.4e38, 2.0 ** 126):
        got, want, _ = _append(x, x, np.arange(64), 4, g, 1.0)
        _same(got, want)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append_quotients_beside_the_border(dtype):
    """Scales one fp32 step to either side of one that makes some |x| exactly half-way between
    two codes, or the largest of a block half-way between two block scales."""
    t, rng = TORCH[dtype], np.random.default_rng(3)
    for trial in range(60):
        x = torch.randn((4, 1, 64), generator=torch.Generator().manual_seed(trial)).to(t)
        v = x.double().numpy().reshape(-1, 16)
        top = np.abs(v).max(1)
        row = int(rng.integers(0, len(v)))
        if trial % 2:
            s = float(rng.integers(8, 16)) * 2.0 ** int(rng.integers(-3, 4))
            pairs = [(a, h) for a in np.abs(v[row]) for h in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)]
            # the scale g that puts a on h s g with this block's top at about 6 s g
            a, h = min(pairs, key=lambda p: abs(p[0] / top[row] - p[1] / 6))
            g = np.float32(a / (h * s))
        else:
            g = np.float32(top[row] / (6 * (rng.integers(8, 16) + 0.5)))
        for step in (np.float32(0), g, np.float32(np.inf)):
            k = np.nextafter(g, step, dtype=np.float32)
            got, want, _ = _append(x.to(DEV), x.to(DEV), np.arange(4), 1, float(k), 1.0)
            _same(got, want)


def test_append_slots_outside():
    x = torch.randn((6, 1, 64), generator=torch.Generator().manual_seed(1)).half().to(DEV)
    got, want, err = _append(x, x, np.array([3, -1, 32, 31, 1 << 30, 0]), 2)
    _same(got, want)
    assert err == pa.PA_DEVERR_SLOT


# ------------------------------------------------------------------ decode

def _decode(dtype, size, kv_heads, group, lens, mode="v2", q_len=None, window=-1, cap=0.0, alibi=False, seed=0, static=False,
            dynamic=False, counters=False, graph=False, ks=0.0019, vs=0.0023, scale=None, ready=False):
    rng, gen = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    n, heads = len(lens), kv_heads * group
    own = [-(-x // 16) for x in lens]
    ids = rng.permutation(sum(own) + 2)
    table = np.full((n, max(max(own), 1)), ids[-1])
    at = np.concatenate([[0], np.cumsum(own)])
    caches = []
    for g in (ks, vs):
        c = pages4(len(ids), kv_heads, size, 0x7f)  # places that no token has: NaN
        slots = []
        for s in range(n):
            table[s, :own[s]] = ids[at[s]:at[s + 1]]
            slots += [table[s, t // 16] * 16 + t % 16 for t in range(lens[s])]
        rows = torch.randn((len(slots), kv_heads, size), generator=gen).half().double().numpy()
        caches.append(store4(c, rows, slots, g))
    k, v = (sequences(values4(c, g), table, lens) for c, g in zip(caches, (ks, vs)))
    rows = sum(q_len) if q_len else n
    start = np.concatenate([[0], np.cumsum(q_len)]) if q_len else np.arange(n + 1)
    q = torch.randn((rows, heads, size), generator=gen).to(TORCH[dtype])
    slopes = np.array([2.0 ** (-8 * (i + 1) / heads) for i in range(heads)], dtype=np.float32) if alibi else None
    top = max(max(lens), 1)
    out, err = torch.full((rows, heads, size), 7.0, dtype=TORCH[dtype], device=DEV), _int([0])
    scale = size ** -0.5 if scale is None else scale
    kw = dict(num_kv_heads=kv_heads, scale=scale, max_seq_len=top, layout="nhd", kv_dtype="e2m1", k_scale=ks, v_scale=vs,
              metadata_ready=ready, window_left=window, softcap=cap, alibi_slopes=None if slopes is None else torch.from_numpy(slopes).to(DEV), dev_error=err)
    if q_len:
        kw.update(query_start=_int(start), max_query_len=max(q_len))
    if dynamic:
        kw.update(seq_lens_host=np.array(lens, dtype=np.int32))
    ws = pa.alloc_workspace(n, heads, size, top, DEV, num_query_tokens=rows if q_len else None,
                            num_kv_heads=kv_heads if counters else None, tile_counters=dynamic)
    args = (out, q.to(DEV), *(torch.from_numpy(c).to(DEV) for c in caches), _int(table), _int(lens))
    if static:
        pa.pa_decode_static_workspace(*args, **kw)
    else:
        pa.pa_decode(*args, mode=mode, **kw, **ws)
        if graph:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                pa.pa_decode(*args, mode=mode, **kw, **ws)
            out.fill_(7.0)
            g.replay()
            g.replay()
    torch.cuda.synchronize()
    assert int(err) == 0
    want = attention(q.double().numpy(), k, v, lens, start, group, scale, cap, slopes, window)
    got = out.double().cpu().numpy()
    absolute, relative = TOL[dtype]
    assert np.all(np.abs(got - want) <= absolute + relative * np.abs(want)), np.abs(got - want).max()
    return ws, k, q


@pytest.mark.parametrize("mode", ["v1", "v2"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size,kv_heads,group", [(64, 2, 2), (128, 2, 7), (128, 1, 8), (64, 1, 1), (128, 2, 12), (64, 2, 16), (128, 1, 16)])
def test_decode(size, kv_heads, group, dtype, mode):
    _decode(dtype, size, kv_heads, group, [1, 15, 16, 17, 0, 300, 513, 1029], mode)


@pytest.mark.parametrize("mode", ["v1", "v2"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size,group,most", [(64, 2, 4), (128, 4, 4), (128, 1, 16), (128, 2, 3)])
def test_decode_several_tokens(size, group, most, dtype, mode):
    lens, q_len = [most, 2, 33, 530, 1030], [most, 2, most - 1, most, 2]
    for window in (-1, 40):
        _decode(dtype, size, 2, group, lens, mode, q_len, window, cap=20.0 if window < 0 else 0.0, alibi=window < 0)


@pytest.mark.parametrize("mode", ["v1", "v2"])
@pytest.mark.parametrize("window,cap,alibi", [(-1, 30.0, True), (0, 0.0, False), (100, 0.0, True), (600, 5.0, False)])
def test_decode_window_softcap_alibi(window, cap, alibi, mode):
    for dtype, size, group in (("f16", 128, 7), ("bf16", 64, 3)):
        _decode(dtype, size, 2, group, [5, 40, 700, 1037], mode, None, window, cap, alibi)


def test_decode_schedules_merges_and_replays():
    _decode("f16", 128, 4, 7, [900] * 6, counters=True, graph=True)
    _decode("bf16", 128, 8, 4, [3000, 40, 1, 2000, 700], mode="auto", dynamic=True, graph=True)
    _decode("f16", 64, 2, 4, [300] * 40, mode="auto", graph=True)
    _decode("f16", 128, 2, 7, [700, 1300], static=True)
    _decode("f16", 128, 4, 7, [900] * 6, graph=True, ready=True)
    _decode("bf16", 64, 8, 2, [3000, 40, 1, 2000, 700], mode="auto", dynamic=True, graph=True, ready=True)


@pytest.mark.parametrize("scale", [-0.11, 0.0, 1e-33, 2.0])
def test_decode_at_any_logit_scale(scale):
    _decode("f16", 64, 2, 3, [300, 700], scale=scale)
    _decode("bf16", 128, 1, 12, [5, 40], "v1", [1, 1], scale=scale)


def test_a_scale_of_one_by_default():
    _decode("f16", 128, 2, 4, [100, 200], ks=1.0, vs=1.0)


def test_blocks_beyond_four_gigabytes():
    """Append, decode, weights and compaction of pages whose places pass 32 bits."""
    blocks, heads, size, n = 520000, 8, 128, 40
    gen = torch.Generator().manual_seed(8)
    kc, vc = (torch.zeros((blocks, heads, 9 * size), dtype=torch.uint8, device=DEV) for _ in range(2))
    assert kc.numel() > 1 << 32
    far, near = np.array([blocks - 1, blocks - 7, blocks - 3]), np.array([1, 5, 2])
    rows = [torch.randn((n, heads, size), generator=gen).half().to(DEV) for _ in range(2)]
    q = torch.randn((1, heads, size), generator=gen).half().to(DEV)
    kept = torch.arange(0, n, 2, dtype=torch.int32, device=DEV).expand(1, heads, -1).contiguous()
    results = []
    for pages in (far, near):
        slots = pages[np.arange(n) // 16] * 16 + np.arange(n) % 16
        pa.pa_append_kv(*rows, kc, vc, _int(slots), layout="nhd", kv_dtype="e2m1", k_scale=0.0019, v_scale=0.0019)
        out, ws = torch.empty_like(q), pa.alloc_workspace(1, heads, size, n, DEV)
        kw = dict(num_kv_heads=heads, scale=size ** -0.5, max_seq_len=n, layout="nhd", kv_dtype="e2m1", k_scale=0.0019)
        table, lens = _int(pages[None]), _int([n])
        pa.pa_decode(out, q, kc, vc, table, lens, mode="v2", v_scale=0.0019, **kw, **ws)
        scores = torch.zeros((blocks, heads, 16), device=DEV)
        pa.pa_add_weights(scores, q, kc, table, lens, ws["exp_sums"], ws["max_logits"], **kw)
        seen = scores[torch.from_numpy(pages).to(DEV)].clone()
        pa.pa_compact_kv(kc, vc, table, kept, _int([n // 2]), scores=scores, layout="nhd", kv_dtype="e2m1")
        at = torch.from_numpy(pages).to(DEV)
        results.append((out, seen, kc[at].clone(), vc[at].clone(), scores[at].clone()))
        assert abs(float(seen.sum()) - heads) < 1e-3  # a whole softmax for every head
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.parametrize("mode,group", [("v1", 4), ("v2", 4), ("v2", 12)])
def test_a_withheld_page_times_out(mode, group):
    """The bounded waits of the 4-bit kernels: a page that never comes ends the call with an error."""
    from paged_kv_attention_v2_gb300 import _abi
    lib = _abi.load()
    gen, size, kv_heads = torch.Generator().manual_seed(2), 128, 2
    caches = [torch.randint(0, 256, (130, kv_heads, 9 * size), generator=gen, dtype=torch.uint8) for _ in range(2)]
    for c in caches:
        c[:, :, 8 * size:] = 0x38  # scales of one
    caches = [c.to(DEV) for c in caches]
    q = torch.randn((3, kv_heads * group, size), generator=gen).half().to(DEV)
    out, err = torch.zeros_like(q), _int([0])
    ws = pa.alloc_workspace(3, kv_heads * group, size, 1300, DEV)
    call = lambda: pa.pa_decode(out, q, *caches, _int(np.arange(246).reshape(3, 82) % 130), _int([700, 1300, 90]), mode=mode,  # noqa: E731
                                num_kv_heads=kv_heads, scale=0.05, max_seq_len=1300, layout="nhd", kv_dtype="e2m1", dev_error=err, **ws)
    call()
    want = out.clone()
    assert int(err) == 0 and torch.isfinite(want).all()
    assert lib.pa_debug_withhold_page(1, 50_000_000) == 0  # 50 ms per wait
    try:
        call()
        torch.cuda.synchronize()
    finally:
        assert lib.pa_debug_withhold_page(0, 0) == 0
    assert int(err) & pa.PA_DEVERR_TIMEOUT
    err.zero_()
    out.zero_()
    call()
    assert int(err) == 0 and torch.equal(out, want)


def test_a_query_beyond_fp16_is_clamped_and_reported():
    c = torch.full((1, 1, 576), 0x38, dtype=torch.uint8, device=DEV)
    ws = pa.alloc_workspace(1, 1, 64, 16, DEV)
    for value, flagged in ((65280.0, False), (65536.0, True), (-1e30, True), (float("inf"), True)):
        q = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device=DEV)
        q[0, 0, 5] = value
        out, err = torch.empty_like(q), _int([0])
        pa.pa_decode(out, q, c, c, _int([[0]]), _int([9]), num_kv_heads=1, scale=1e-6, max_seq_len=16, layout="nhd", kv_dtype="e2m1",
                     dev_error=err, **ws)
        assert int(err) == (8 if flagged else 0), value  # PA_DEVERR_QUERY_RANGE
        assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,size,ctas", [(28, 4, 128, 3), (64, 4, 128, 2), (8, 2, 64, 3)])
def test_plan(dtype, heads, kv_heads, size, ctas):
    """pa_plan tells of a 4-bit call what it launches."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for lens, merged in (([4096] * 32, False), ([1500, 1100], True)):
        q = torch.zeros((len(lens), heads, size), dtype=TORCH[dtype], device=DEV)
        k = torch.zeros((4, kv_heads, 9 * size), dtype=torch.uint8, device=DEV)
        ws = pa.alloc_workspace(len(lens), heads, size, max(lens), DEV, num_kv_heads=kv_heads)
        g = pa.plan_for(q, q, k, k, torch.zeros((len(lens), 256), dtype=torch.int32, device=DEV),
                        torch.zeros(len(lens), dtype=torch.int32, device=DEV), num_kv_heads=kv_heads, scale=0.1, max_seq_len=max(lens),
                        layout="nhd", mode="v2", kv_dtype="e2m1", **ws)
        tiles = kv_heads * len(lens) * -(-max(lens) // 512)
        assert (g["mode"], g["ctas_per_sm"], g["merge_in_kernel"], g["kernels"]) == ("v2", ctas, merged, 1 if merged else 2)
        assert 1 <= g["grid"] <= min(tiles, ctas * sms)
