"""GPU tests of pa_add_weights, pa_select_tokens and pa_compact_kv against their
statements in 64 bits (weights), whole numbers (selection) and bits (compaction)."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import paged_kv_attention_v2_gb300 as pa  # noqa: E402
from cache_ref import cache_shapes  # noqa: E402
from short_ref import compact_ref, pages4, row_weights, select_ref, sequences, store4, values4  # noqa: E402

DEV = "cuda:0"
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
         "e5m2": torch.float8_e5m2}


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _table(rng, lens, spare=2):
    own = [-(-x // 16) for x in lens]
    ids = rng.permutation(sum(own) + spare)
    table = np.full((len(lens), max(max(own), 1)), ids[-1])
    at = np.concatenate([[0], np.cumsum(own)])
    for s in range(len(lens)):
        table[s, :own[s]] = ids[at[s]:at[s + 1]]
    return table, len(ids)


# ------------------------------------------------------------------ weights

# A logit's sum of `size` products of about unit normals, times 1 / sqrt(size): its terms add up to about 7 at size
# 128, so 1e-4 is over a hundred half steps of fp32 of that; the level's and the exponential's own roundings are
# a few 2^-23.  A weight is off by that relative to itself, and so is a sum of weights.  With ALiBi the given
# maxima are rounded numbers of up to slope x position = 1100: half a step more, 6e-5.
REL, REL_ALIBI = 2e-4, 3e-4
# The maxima of a decode have been moved from the last token's position to the sequence's first: products and sums of up
# to slope x position = 1350, four roundings of 6e-5.
REL_DECODE_ALIBI = 5e-4


def _weights(dtype, kv, layout, size, kv_heads, group, lens, q_len=None, window=-1, cap=0.0, alibi=False, decay=1.0, seed=0,
             from_decode=False, graph=False):
    rng, gen = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    n, heads = len(lens), kv_heads * group
    table, blocks = _table(rng, lens)
    ks = {None: 1.0, "e2m1": 0.0019}.get(kv, 2.0 ** -5)
    rows = torch.randn((blocks, kv_heads, 16, size), generator=gen)
    if kv == "e2m1":
        c = pages4(blocks, kv_heads, size)
        flat = rows.half().double().numpy().transpose(0, 2, 1, 3).reshape(-1, kv_heads, size)
        c = store4(c, flat, np.arange(blocks * 16), ks)
        cache, values = torch.from_numpy(c).to(DEV), values4(c, ks)
    else:
        c = (rows / ks).to(TORCH[kv or dtype])
        values = c.double().numpy() * ks
        if layout == "split":
            x = 16 // c.element_size()
            c = c.unflatten(3, (size // x, x)).permute(0, 1, 3, 2, 4)
        cache = c.contiguous().to(DEV)
    nrows = sum(q_len) if q_len else n
    start = np.concatenate([[0], np.cumsum(q_len)]) if q_len else np.arange(n + 1)
    q = torch.randn((nrows, heads, size), generator=gen).to(TORCH[dtype])
    slopes = np.array([2.0 ** (-8 * (i + 1) / heads) for i in range(heads)], dtype=np.float32) if alibi else None
    top = max(max(lens), 1)
    parts = max(1, -(-top // 512))
    m, e = np.full((nrows, heads, parts), -np.inf), np.zeros((nrows, heads, parts))
    k, qd = sequences(values, table, lens), q.double().numpy()
    scores = rng.random((blocks, kv_heads, 16)).astype(np.float32)
    want = scores.astype(np.float64)
    for s, length in enumerate(lens):
        qn = start[s + 1] - start[s]
        added = np.zeros((length, kv_heads))
        for r in range(start[s], start[s + 1]):
            pos = length - (start[s + 1] - r)
            if pos < 0:
                continue
            lo = max(0, pos - window) if window >= 0 else 0
            for h in range(heads):
                slope = 0.0 if slopes is None else float(slopes[h])
                w = row_weights(qd[r, h], k[s][:, h // group], size ** -0.5, lo, pos, cap, slope)
                added[lo:pos + 1, h // group] += w
                z = size ** -0.5 * k[s][lo:pos + 1, h // group] @ qd[r, h]
                z = (cap * np.tanh(z / cap) if cap > 0 else z) + slope * np.arange(lo, pos + 1)
                for p in range(lo // 512, pos // 512 + 1):
                    zp = z[max(p * 512 - lo, 0):max((p + 1) * 512 - lo, 0)]
                    m[r, h, p] = np.float32(zp.max())
                    e[r, h, p] = np.exp(zp - m[r, h, p]).sum()
        for t in range(length):
            b, o = table[s, t // 16], t % 16
            fresh = decay == 0 or t >= length - qn
            want[b, :, o] = added[t] if fresh else np.float64(np.float32(decay)) * want[b, :, o] + added[t]
            if fresh:
                scores[b, :, o] = np.nan  # whatever a new token's slot holds
    real = lambda a: torch.from_numpy(a.astype(np.float32)).to(DEV)  # noqa: E731
    sums, most, got, err = real(e), real(m), torch.from_numpy(scores).to(DEV), _int([0])
    kw = dict(num_kv_heads=kv_heads, scale=size ** -0.5, max_seq_len=top, layout=layout, kv_dtype=kv, k_scale=ks,
              window_left=window, softcap=cap, alibi_slopes=None if slopes is None else torch.from_numpy(slopes).to(DEV), dev_error=err)
    if q_len:
        kw.update(query_start=_int(start), max_query_len=max(q_len))
    qg, tg, lg = q.to(DEV), _int(table), _int(lens)
    if from_decode:
        ws = pa.alloc_workspace(n, heads, size, top, DEV, num_query_tokens=nrows if q_len else None, num_kv_heads=kv_heads)
        raw = cache.view(torch.uint8) if kv else cache
        pa.pa_decode(torch.empty_like(qg), qg, raw, raw if layout == "nhd" else raw.reshape(blocks, kv_heads, size, 16), tg, lg,
                     mode="v2", v_scale=1.0, **kw, **ws)
        sums, most = ws["exp_sums"], ws["max_logits"]
    call = lambda: pa.pa_add_weights(got, qg, cache, tg, lg, sums, most, decay=decay, **kw)  # noqa: E731
    if graph:
        saved = got.clone()
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        got.copy_(saved)
        g.replay()
    else:
        call()
    torch.cuda.synchronize()
    assert int(err) == 0
    out = got.double().cpu().numpy()
    rel = REL if not alibi else REL_DECODE_ALIBI if from_decode else REL_ALIBI
    ok = np.abs(out - want) <= rel * np.abs(want) + 1e-30
    assert ok.all(), (np.argwhere(~ok)[:4], out[~ok][:4], want[~ok][:4])


KINDS = [("f32", None, "split"), ("f32", None, "nhd"), ("f16", None, "split"), ("f16", None, "nhd"), ("bf16", None, "split"),
         ("bf16", None, "nhd"), ("f16", "e4m3", "split"), ("bf16", "e4m3", "nhd"), ("bf16", "e5m2", "split"), ("f16", "e5m2", "nhd"),
         ("f16", "e2m1", "nhd"), ("bf16", "e2m1", "nhd")]
LENS = [1, 15, 16, 17, 0, 300, 513, 1029]


@pytest.mark.parametrize("dtype,kv,layout", KINDS)
@pytest.mark.parametrize("size,kv_heads,group", [(64, 2, 2), (128, 2, 7), (128, 1, 8), (64, 1, 1), (128, 2, 12), (64, 2, 16), (128, 1, 16)])
def test_weights(size, kv_heads, group, dtype, kv, layout):
    _weights(dtype, kv, layout, size, kv_heads, group, LENS)


@pytest.mark.parametrize("dtype,kv,layout", KINDS)
@pytest.mark.parametrize("size,group,most", [(64, 2, 4), (128, 4, 4), (128, 1, 16)])
def test_weights_of_several_tokens(size, group, most, dtype, kv, layout):
    lens, q_len = [most, 2, 33, 530, 1030, 2], [most, 2, most - 1, most, 0, most]
    for window, decay in ((-1, 1.0), (40, 0.9)):
        _weights(dtype, kv, layout, size, 2, group, lens, q_len, window, cap=20.0 if window < 0 else 0.0, alibi=window < 0, decay=decay)


@pytest.mark.parametrize("window,cap,alibi,decay", [(-1, 30.0, True, 0.0), (0, 0.0, False, 1.0), (100, 0.0, True, 0.5), (600, 5.0, False, 0.0)])
def test_weights_window_softcap_alibi_decay(window, cap, alibi, decay):
    for dtype, kv, layout, size, group in (("f16", None, "split", 128, 7), ("bf16", "e4m3", "nhd", 64, 3), ("f32", None, "nhd", 64, 2)):
        _weights(dtype, kv, layout, size, 2, group, [5, 40, 700, 1037], None, window, cap, alibi, decay)


def test_weights_from_the_statistics_of_a_decode():
    _weights("f16", None, "split", 128, 2, 7, [40, 700, 2000], from_decode=True)
    _weights("bf16", "e2m1", "nhd", 128, 2, 4, [40, 700, 2000], from_decode=True)
    _weights("bf16", "e4m3", "nhd", 64, 2, 2, [40, 700, 2000], [4, 1, 3], from_decode=True, decay=0.0, graph=True)
    for lens in ([40, 700, 2000], [900] * 30):  # merged in the partition kernel, and by the reduce kernel
        _weights("f16", None, "split", 128, 2, 7, lens, alibi=True, cap=20.0, from_decode=True)
        _weights("bf16", "e2m1", "nhd", 64, 2, 2, lens, window=600, from_decode=True)
        _weights("f32", None, "nhd", 64, 2, 4, lens, from_decode=True)


def test_weights_of_long_sequences_in_longer_tiles():
    _weights("f16", "e2m1", "nhd", 64, 2, 1, [9000, 30000], graph=True)
    _weights("bf16", None, "split", 64, 16, 1, [5000] * 12)


def test_weights_skip_pages_out_of_range():
    q = torch.randn(1, 1, 64, device=DEV).half()
    k = torch.randn(3, 1, 16, 64, device=DEV).half()
    scores = torch.full((3, 1, 16), 5.0, device=DEV)
    err = _int([0])
    one = torch.ones(1, 1, 1, device=DEV)
    pa.pa_add_weights(scores, q, k, _int([[1, 7, -1]]), _int([40]), one, one, num_kv_heads=1, scale=0.1, max_seq_len=48,
                      layout="nhd", dev_error=err)
    assert int(err) == pa.PA_DEVERR_BLOCK_ID
    s = scores.cpu()
    assert (s[0] == 5).all() and (s[2] == 5).all() and (s[1] > 5).all()


@pytest.mark.parametrize("kv", [None, "e2m1"])
def test_weights_do_not_look_at_pages_before_the_window_unless_they_fade(kv):
    """300 tokens, the last 21 within the window: pages 0 to 16 have no token in it."""
    q = torch.randn(1, 1, 64, device=DEV).half()
    k = torch.zeros(20, 1, 9 * 64, dtype=torch.uint8, device=DEV) if kv else torch.zeros(20, 1, 16, 64, device=DEV).half()
    one = torch.ones(1, 1, 1, device=DEV)
    table = np.arange(20)
    table[3] = 99
    for decay, bit in ((1.0, 0), (0.5, pa.PA_DEVERR_BLOCK_ID)):
        scores = torch.full((20, 1, 16), 5.0, device=DEV)
        scores[6, 0, 2] = float("nan")
        err = _int([0])
        pa.pa_add_weights(scores, q, k, _int(table[None]), _int([300]), one, torch.zeros_like(one), num_kv_heads=1, scale=0.1, max_seq_len=320,
                          layout="nhd", kv_dtype=kv, window_left=20, decay=decay, dev_error=err)
        assert int(err) == bit
        s = scores.cpu().flatten()
        assert (s[300:] == 5).all() and s[299] == 1 and torch.isnan(s[98])  # zero keys: logits 0, weights exp(0) / 1
        assert (s[279:299] == 5 * decay + 1).all() and (s[48:64] == 5).all()
        rest = torch.cat([s[:48], s[64:98], s[99:279]])
        assert (rest == 5 * decay).all()


# ------------------------------------------------------------------ selection

def _select(lens, heads, budgets, sink, recent, scores=None, seed=0, graph=False):
    rng = np.random.default_rng(seed)
    table, blocks = _table(rng, lens)
    if scores is None:
        scores = rng.random((blocks, heads, 16)).astype(np.float32) ** 6
        scores[rng.random(scores.shape) < 0.1] = 0.125  # ties
    else:
        scores = scores(rng, (blocks, heads, 16)).astype(np.float32)
    top, most = max(max(lens), 1), max(max(budgets), 1)
    kept, new, err = torch.full((len(lens), heads, most), -9, dtype=torch.int32, device=DEV), _int(np.full(len(lens), -9)), _int([0])
    args = (kept, new, torch.from_numpy(scores).to(DEV), _int(table), _int(lens), _int(budgets))
    kw = dict(max_seq_len=top, sink=sink, recent=recent, dev_error=err)
    pa.pa_select_tokens(*args, **kw)
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.pa_select_tokens(*args, **kw)
        kept.fill_(-9)
        g.replay()
    torch.cuda.synchronize()
    assert int(err) == 0
    want, lens_want = select_ref(scores, table, lens, budgets, sink, recent, most, -9)
    assert np.array_equal(new.cpu().numpy(), lens_want)
    got = kept.cpu().numpy()
    assert np.array_equal(got, want), np.argwhere(got != want)[:4]


@pytest.mark.parametrize("sink,recent", [(0, 0), (4, 0), (0, 16), (4, 64), (1000, 1000)])
def test_select(sink, recent):
    lens = [1, 15, 16, 17, 0, 300, 513, 1029, 4096, 5000]
    for budgets in ([10] * 10, [0] * 10, [1, 15, 15, 9, 0, 299, 17, 1029, 4000, 77], [5000] * 10):
        _select(lens, 3, budgets, sink, recent)


@pytest.mark.parametrize("n,seqs,heads", [(4097, 2, 1), (10000, 4, 2), (40000, 2, 4), (70001, 1, 3), (170000, 1, 1), (340000, 1, 2)])
def test_select_long(n, seqs, heads):
    rng = np.random.default_rng(n)
    for share in (0.02, 0.5, 0.99):
        lens = [n] + [int(x) for x in rng.integers(1, n, seqs - 1)]
        _select(lens, heads, [max(1, int(n * share))] * seqs, 4, 100, seed=n, graph=share == 0.5)


def test_select_scores_of_every_kind():
    def odd(rng, shape):
        pick = np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 3.4e38, -3.4e38, 1.0, -1.0], dtype=np.float32)
        return pick[rng.integers(0, len(pick), shape)]
    for budget in (1, 7, 100, 333, 699):
        _select([700, 650, 3], 2, [budget] * 3, 0, 0, odd)
    _select([3000], 2, [1500], 0, 0, lambda rng, s: np.zeros(s))          # all the same
    _select([3000], 2, [1500], 2, 2, lambda rng, s: np.full(s, np.nan))
    _select([50000] * 3, 1, [777] * 3, 0, 0, lambda rng, s: (rng.integers(0, 3, s) * 0.5))


def test_select_out_of_range():
    scores = torch.rand(4, 1, 16, device=DEV)
    kept, new, err = torch.full((2, 1, 8), -9, dtype=torch.int32, device=DEV), _int([0, 0]), _int([0])
    pa.pa_select_tokens(kept, new, scores, _int([[0, 1], [2, 3]]), _int([20, 90]), _int([8, 99]), max_seq_len=32, dev_error=err)
    assert int(err) == pa.PA_DEVERR_SEQ_LEN and new.tolist() == [8, 8]
    assert (kept[1, 0].cpu().diff() > 0).all() and int(kept.max()) < 32
    err.zero_()
    pa.pa_select_tokens(kept, new, scores, _int([[0, 55], [2, -3]]), _int([20, 31]), _int([8, 8]), max_seq_len=32, dev_error=err)
    assert int(err) == pa.PA_DEVERR_BLOCK_ID
    assert (kept.cpu() < 16).all()  # those without a score go first


# ------------------------------------------------------------------ compaction

def _compact(dtype, layout, k_heads, k_size, v_heads, v_size, kv_heads, lens, choose, scores=True, seed=0, graph=False):
    rng = np.random.default_rng(seed)
    table, blocks = _table(rng, lens)
    kv = dtype if dtype in ("e4m3", "e5m2", "e2m1") else None
    if dtype == "e2m1":
        shapes, bits = ((blocks, k_heads, 9 * k_size), (blocks, v_heads, 9 * v_size)), np.uint8
    else:
        width = TORCH[dtype].itemsize
        shapes, bits = cache_shapes(blocks, k_heads, k_size, v_heads, v_size, layout, width), {1: np.uint8, 2: np.int16, 4: np.int32}[width]
    caches = [rng.integers(np.iinfo(bits).min, np.iinfo(bits).max, s, dtype=bits, endpoint=True) for s in shapes]
    sc = rng.random((blocks, kv_heads, 16)).astype(np.float32)
    new, kept = choose(rng, lens, kv_heads)
    gpu = [torch.from_numpy(c.copy()).to(DEV) for c in caches]
    view = [g if dtype == "e2m1" else g.view(TORCH[dtype]) for g in gpu]
    sg, err = torch.from_numpy(sc.copy()).to(DEV) if scores else None, _int([0])
    call = lambda: pa.pa_compact_kv(*view, _int(table), kg, ng, scores=sg, layout=layout, kv_dtype=kv, dev_error=err)  # noqa: E731
    kg, ng = _int(kept), _int(new)
    if graph:
        tg = _int(table)
        args = lambda: pa.pa_compact_kv(*view, tg, kg, ng, scores=sg, layout=layout, kv_dtype=kv, dev_error=err)  # noqa: E731
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            args()
        g.replay()
    else:
        call()
    torch.cuda.synchronize()
    assert int(err) == 0
    want = compact_ref(caches, sc if scores else None, table, kept, new, layout, kv_heads, dtype == "e2m1")
    for g, w in zip(gpu + ([sg] if scores else []), want):
        same = g.cpu().numpy().view(np.uint8) == w.view(np.uint8)
        assert same.all(), np.argwhere(~same)[:4]


def _random(share):
    def choose(rng, lens, heads):
        new = [int(n * share) if n else 0 for n in lens]
        kept = np.full((len(lens), heads, max(max(new), 1)), -1)
        for s, n in enumerate(lens):
            for h in range(heads):
                kept[s, h, :new[s]] = np.sort(rng.permutation(n)[:new[s]])
        return new, kept
    return choose


def _front(drop):
    """All but `drop` tokens after the first few."""
    def choose(rng, lens, heads):
        new = [max(n - drop, 0) for n in lens]
        kept = np.full((len(lens), heads, max(max(new), 1)), -1)
        for s in range(len(lens)):
            for h in range(heads):
                first = min(new[s], 3 + h)
                kept[s, h, :new[s]] = np.concatenate([np.arange(first), np.arange(first, new[s]) + drop])
        return new, kept
    return choose


LONG = [1, 16, 17, 0, 300, 513, 1100, 2600]


@pytest.mark.parametrize("dtype,layout", [("f32", "split"), ("f32", "nhd"), ("f16", "split"), ("f16", "nhd"), ("bf16", "split"), ("bf16", "nhd"),
                                          ("e4m3", "split"), ("e5m2", "nhd"), ("e2m1", "nhd")])
@pytest.mark.parametrize("k_heads,k_size,v_heads,v_size,kv_heads", [(2, 128, 2, 128, 2), (1, 64, 1, 64, 1), (4, 64, 2, 128, 2), (3, 64, 3, 128, 3),
                                                                    (4, 128, 2, 256, 2)])
def test_compact(k_heads, k_size, v_heads, v_size, kv_heads, dtype, layout):
    if dtype == "e2m1" and v_size == 256:
        pytest.skip("refused: 4-bit heads of 256")
    for i, choose in enumerate((_random(0.5), _random(0.06), _random(0.97), _front(1), _front(17))):
        _compact(dtype, layout, k_heads, k_size, v_heads, v_size, kv_heads, LONG, choose, scores=i % 2 == 0, seed=i, graph=i == 2)


def test_compact_many_times_is_the_same():
    """A race between a chunk's loads and stores would show now and then."""
    for seed in range(30):
        _compact("f16", "split", 2, 128, 2, 128, 2, [3000, 2900, 2800], _front(1 + seed), seed=seed)
        _compact("bf16", "nhd", 2, 64, 2, 64, 2, [3000, 2900, 2800], _front(1 + 16 * seed), seed=seed)


def test_compact_all_stay():
    def same(rng, lens, heads):
        kept = np.tile(np.arange(max(lens)), (len(lens), heads, 1))
        return lens, kept
    _compact("f16", "nhd", 2, 64, 2, 64, 2, [300, 40], same)


def test_compact_reports_what_it_does_not_move():
    k = torch.randn(3, 1, 16, 64, device=DEV).half()
    before, err = k.clone(), _int([0])
    for kept, bit in (([[[0, 5, 5, 9]]], pa.PA_DEVERR_SLOT), ([[[1, 0, 30, 40]]], pa.PA_DEVERR_SLOT), ([[[0, 1, 2, 4000]]], pa.PA_DEVERR_SLOT)):
        err.zero_()
        pa.pa_compact_kv(k, k.clone(), _int([[0, 1, 2]]), _int(kept), _int([4]), layout="nhd", dev_error=err)
        assert int(err) == bit
        assert torch.equal(k[0, 0, 4:], before[0, 0, 4:]) and torch.equal(k[1:], before[1:])
    err.zero_()
    pa.pa_compact_kv(k, k.clone(), _int([[0, 77, -1]]), _int([[[0, 20]]]), _int([2]), layout="nhd", dev_error=err)
    assert int(err) == pa.PA_DEVERR_BLOCK_ID
    err.zero_()
    pa.pa_compact_kv(k, k.clone(), _int([[0, 1, 2]]), _int([[[0, 1]]]), _int([9]), layout="nhd", dev_error=err)
    assert int(err) == pa.PA_DEVERR_SEQ_LEN


@pytest.mark.parametrize("dtype,layout", [("f32", "split"), ("f16", "split"), ("e4m3", "split"), ("bf16", "nhd"), ("e5m2", "nhd"), ("e2m1", "nhd")])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_compact_moves_the_others(dtype, layout, seed):
    """Entries that are refused, and pages that are not there, among ones that move: only those places stay as they were."""
    rng = np.random.default_rng(seed)
    n, heads, size, blocks = 1100, 2, 64, 100
    pages = -(-n // 16)
    table = rng.permutation(blocks)[:pages]
    kept = np.stack([np.sort(rng.permutation(n)[:n - 14 - 300 * seed]) if seed else np.concatenate([np.arange(5), np.arange(5, n - 9) + 9])
                     for _ in range(heads)])
    count = kept.shape[1]
    bad = rng.random(kept.shape) < 0.1
    kept = np.where(bad, np.where(rng.random(kept.shape) < 0.5, np.arange(count) - 1, 16 * pages + 5), kept)
    away = rng.permutation(pages)[:3]
    table[away] = (blocks, -1, blocks + 70)
    elem = {"f32": 4, "f16": 2, "bf16": 2}.get(dtype, 1)
    kv = dtype if elem == 1 else None
    shapes = (((blocks, heads, 9 * size),) * 2 if dtype == "e2m1" else cache_shapes(blocks, heads, size, heads, size, layout, elem))
    bits = {1: np.uint8, 2: np.int16, 4: np.int32}[elem]
    caches = [rng.integers(np.iinfo(bits).min, np.iinfo(bits).max, s, dtype=bits, endpoint=True) for s in shapes]
    ok = np.zeros(kept.shape, dtype=bool)
    for h in range(heads):
        for i in range(count):
            k = kept[h, i]
            if k >= i and k > (kept[h, i - 1] if i else -1) and k < 16 * pages:
                ok[h, i] = k == i or (0 <= table[k // 16] < blocks and 0 <= table[i // 16] < blocks)

    def move(x, w, token):  # token(x, block, head, t): that token's elements of a cache, in place
        for h in range(heads):
            for i in np.flatnonzero(ok[h]):
                if kept[h, i] != i:
                    token(w, table[i // 16], h, i % 16)[...] = token(x, table[kept[h, i] // 16], h, kept[h, i] % 16)
        return w
    rows = lambda x, b, h, t: x[b, h, t]  # noqa: E731
    if dtype == "e2m1":
        places = [lambda x, b, h, t: x[b, h, :8 * size].reshape(16, size // 2)[t], lambda x, b, h, t: x[b, h, 8 * size:].reshape(16, size // 16)[t]]
        want = [x.copy() for x in caches]
        for place in places:
            for x, w in zip(caches, want):
                move(x, w, place)
    elif layout == "nhd":
        want = [move(x, x.copy(), rows) for x in caches]
    else:
        want = [move(caches[0], caches[0].copy(), lambda x, b, h, t: x[b, h, :, t]),
                move(caches[1], caches[1].copy(), lambda x, b, h, t: x[b, h, :, t])]
    gpu = [torch.from_numpy(c.copy()).to(DEV) for c in caches]
    view = [g if dtype == "e2m1" else g.view(TORCH[dtype]) for g in gpu]
    err = _int([0])
    pa.pa_compact_kv(*view, _int(table[None]), _int(kept[None]), _int([count]), layout=layout, kv_dtype=kv, dev_error=err)
    torch.cuda.synchronize()
    assert int(err) == pa.PA_DEVERR_SLOT | pa.PA_DEVERR_BLOCK_ID
    for g, w in zip(gpu, want):
        same = g.cpu().numpy() == w
        assert same.all(), np.argwhere(~same)[:4]
