"""GPU tests of pa_build_tables and pa_append_kv: every output against the plain
statements of cache_ref.py, bit for bit (nothing here is rounded but fp8, whose
value is one fp32 product with 1 / scale, rounded by torch's own conversion)."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import paged_kv_attention_v2_gb300 as pa  # noqa: E402
from cache_ref import cache_shapes, make_batch, store_ref, tables_ref  # noqa: E402

DEV = "cuda:0"


def _int(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


class Step:
    """A batch on the GPU with outputs full of marks."""

    def __init__(self, b, rows=None, misaligned=False, in_place=False, counter=True):
        self.b, self.rows = b, b["tokens"] if rows is None else rows
        n = len(b["lens"])
        self.table, self.lens, self.ring, self.state = _int(b["table"]), _int(b["lens"]), _int(b["ring"]), _int(b["state"])
        self.keep, self.start = _int(b["keep"]), _int(b["start"])
        off = 1 if misaligned else 0
        self.slots = torch.full((self.rows + off + 3,), 77, dtype=torch.int32, device=DEV)
        self.positions = torch.full((self.rows + off + 3,), 77, dtype=torch.int32, device=DEV)
        self.view = slice(off, off + self.rows)
        self.new_lens = self.lens if in_place else torch.full((n,), 77, dtype=torch.int32, device=DEV)
        self.new_state = self.state if in_place else torch.full((2,), 77, dtype=torch.int32, device=DEV)
        self.counter = torch.zeros(1, dtype=torch.int32, device=DEV) if counter else None
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call(self, **kw):
        pa.pa_build_tables(self.table, self.lens, self.ring, self.state, self.slots[self.view],
                           max_seq_len=self.b["max_len"], keep_lens=self.keep, query_start=self.start,
                           positions=self.positions[self.view], new_seq_lens=self.new_lens,
                           new_pool_state=self.new_state, done_counter=self.counter, dev_error=self.err, **kw)

    def check(self, err=0):
        torch.cuda.synchronize()
        b = self.b
        table, ring, slots, positions, new, state = tables_ref(b["table"], b["lens"], b["ring"], b["state"], self.rows,
                                                               b["keep"], b["start"])
        assert int(self.err) == err
        for name, got, want in (("table", self.table, table), ("ring", self.ring, ring), ("lens", self.new_lens, new),
                                ("state", self.new_state, state), ("slots", self.slots[self.view], slots),
                                ("positions", self.positions[self.view], positions)):
            got = got.cpu().numpy()
            assert np.array_equal(got, want), (name, np.argwhere(got != want)[:5])
        outside = [i for i in range(self.slots.numel()) if not self.view.start <= i < self.view.stop]
        assert (self.slots[outside] == 77).all() and (self.positions[outside] == 77).all()
        assert self.counter is None or int(self.counter) == 0

    def check_nothing_done(self, err):
        torch.cuda.synchronize()
        b = self.b
        assert int(self.err) == err
        for got, want in ((self.table, b["table"]), (self.ring, b["ring"]), (self.new_lens, b["lens"]),
                          (self.new_state, b["state"])):
            assert np.array_equal(got.cpu().numpy(), want)
        assert (self.slots[self.view] == -1).all() and (self.positions[self.view] == 0).all()


TABLES = [
    # sequences, longest, tokens each, cut, one token each, padding rows
    (1, 1, 1, False, True, 0), (1, 40, 0, False, False, 5), (3, 33, 17, True, False, 0), (32, 4096, 1, False, True, 0),
    (33, 500, 4, True, False, 7), (300, 900, 16, True, False, 100), (1000, 200, 2, True, True, 13),
    (1025, 64, 3, False, False, 1), (4096, 64, 2, True, False, 0), (4097, 48, 2, True, False, 9),
    (9000, 40, 2, True, False, 0), (9000, 30, 1, False, True, 2), (2, 40000, 3, True, False, 0),
    (7, 100, 30000, False, False, 3), (5, 5000, 50000, True, False, 0), (200, 16, 5000, True, False, 0),
]


@pytest.mark.parametrize("n,longest,tokens,cut,single,pad", TABLES)
@pytest.mark.parametrize("counter", [True, False], ids=["many", "one"])
def test_tables(n, longest, tokens, cut, single, pad, counter):
    b = make_batch(n * 7 + tokens, n, longest, tokens, cut=cut, single=single)
    s = Step(b, rows=b["tokens"] + pad, counter=counter)
    s.call()
    s.check()


@pytest.mark.parametrize("n,longest,tokens,single", [(5, 100, 3, False), (64, 300, 1, True), (50, 4000, 3000, False),
                                                     (5000, 40, 2, False)])
def test_tables_in_place_misaligned_and_without_positions(n, longest, tokens, single):
    b = make_batch(11, n, longest, tokens, cut=True, single=single)
    s = Step(b, rows=b["tokens"] + 6, misaligned=True, in_place=True)
    s.call()
    s.check()
    s = Step(b)
    pa.pa_build_tables(s.table, s.lens, s.ring, s.state, s.slots[s.view], max_seq_len=b["max_len"], keep_lens=s.keep,
                       query_start=s.start, done_counter=s.counter)
    s.new_lens, s.new_state = s.lens, s.state  # the defaults: in place
    s.positions[s.view] = _int(tables_ref(b["table"], b["lens"], b["ring"], b["state"], s.rows, b["keep"], b["start"])[3])
    s.check()


def test_tables_many_steps_lose_no_page():
    """Prompts, growth, rejected drafts, ends and new prompts in place, over and over:
    each step as the plain statement has it, and every page owned once or free once."""
    rng = np.random.default_rng(5)
    n, width, blocks = 24, 40, 24 * 40
    lens = np.zeros(n, dtype=np.int64)
    b = dict(table=np.full((n, width), -1, dtype=np.int64), lens=lens, ring=rng.permutation(blocks),
             state=np.array([17, blocks]), keep=None, start=None, max_len=width * 16, tokens=0)
    b["ring"] = np.roll(b["ring"], 17)
    for step in range(60):
        keep = np.maximum(b["lens"] - rng.integers(0, 6, n), 0)
        keep[rng.random(n) < 0.1] = 0
        new = np.where(keep == 0, rng.integers(0, 300, n), rng.integers(0, 8, n))
        new = np.minimum(new, b["max_len"] - keep)
        b.update(keep=keep, start=np.concatenate([[0], np.cumsum(new)]), tokens=int(new.sum()))
        s = Step(b, in_place=True)
        s.call()
        s.check()
        table, ring, _, _, lens, state = tables_ref(b["table"], b["lens"], b["ring"], b["state"], s.rows, keep, b["start"])
        b.update(table=table, ring=ring, lens=lens, state=state)
        owned = [table[i, p] for i in range(n) for p in range(-(-int(lens[i]) // 16))]
        assert sorted(owned + [ring[(state[0] + k) % blocks] for k in range(state[1])]) == list(range(blocks))


@pytest.mark.parametrize("n", [9, 6000])
def test_tables_refuse_as_a_whole(n):
    good = make_batch(2, n, 60, 60, cut=True)

    def with_(**over):
        return {**good, **{k: np.array(v) for k, v in over.items()}}

    def at(a, i, v):
        a = np.array(a)
        a[i] = v
        return a

    lens, keep, start, ml = good["lens"], good["keep"], good["start"], good["max_len"]
    for bad in (with_(lens=at(lens, 4, -1)), with_(lens=at(lens, n - 1, ml + 1)), with_(keep=at(keep, 3, -2)),
                with_(keep=at(keep, 3, lens[3] + 1)), with_(start=at(start, n // 2, start[n // 2 - 1] - 1)),
                with_(start=at(start, n, start[n - 1] + ml + 1)), with_(start=at(start, 0, 1)),
                with_(start=at(start, n, 2 ** 31 - 1)), with_(start=at(start, 2, -2 ** 31))):
        s = Step(bad, rows=good["tokens"] + 4)
        s.call()
        s.check_nothing_done(pa.PA_DEVERR_SEQ_LEN)
    need = int(np.maximum(-(-(keep + np.diff(start)) // 16) - -(-lens // 16), 0).sum())
    assert need > 2
    blocks = len(good["ring"])
    for state in ([3, need - 1], [-1, need], [blocks, need], [0, blocks + 1], [0, -1], [0, blocks]):
        s = Step(with_(state=state), rows=good["tokens"] + 4)
        s.call()
        s.check_nothing_done(pa.PA_DEVERR_POOL)
    s = Step(with_(state=[3, need]))  # just enough
    s.call()
    s.check()


def test_tables_bad_page_ids():
    b = make_batch(8, 6, 100, 20)
    b["ring"][(b["state"][0] + 1) % len(b["ring"])] = len(b["ring"])
    b["ring"][(b["state"][0] + 2) % len(b["ring"])] = -3
    s = Step(b)
    s.call()
    torch.cuda.synchronize()
    table, _, slots, _, _, _ = tables_ref(b["table"], b["lens"], b["ring"], b["state"], s.rows, b["keep"], b["start"])
    assert int(s.err) == pa.PA_DEVERR_BLOCK_ID
    assert np.array_equal(s.table.cpu().numpy(), table)
    bad = (slots < 0) | (slots >= 16 * len(b["ring"]))
    assert bad.any() and np.array_equal(s.slots.cpu().numpy()[:s.rows], np.where(bad, -1, slots))


def test_tables_empty_batch_is_padding():
    b = dict(table=np.zeros((0, 4)), lens=np.zeros(0), keep=None, start=None, ring=np.arange(8), state=np.array([2, 8]),
             max_len=64, tokens=0)
    for start in (None, np.zeros(1)):
        s = Step({**b, "start": start}, rows=5000)
        s.call()
        s.check_nothing_done(0)


def test_tables_graph_and_other_stream():
    b = make_batch(4, 40, 700, 900, cut=True)
    s = Step(b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    s.check()
    s = Step(b)
    table, ring = s.table.clone(), s.ring.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.call()
    for _ in range(3):
        s.table.copy_(table)
        s.ring.copy_(ring)
        s.slots.fill_(77)
        g.replay()
        s.check()


# ------------------------------------------------------------------ append

TYPES = [("f32", None), ("f16", None), ("bf16", None), ("f16", "e4m3"), ("bf16", "e5m2"), ("bf16", "e4m3"), ("f16", "e5m2")]
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
BITS = {1: torch.uint8, 2: torch.int16, 4: torch.int32}


def _quantised(x, kv, scale):
    """Element bits of a row: x itself, or fp8(x * (1 / scale)), beyond the largest value that value."""
    if kv is None:
        return x.cpu().view(BITS[x.element_size()]).numpy()
    q = x.cpu().float() * (torch.tensor(1.0) / torch.tensor(scale, dtype=torch.float32))
    top = torch.finfo(FP8[kv]).max
    return q.clamp(-top, top).to(FP8[kv]).view(torch.uint8).numpy()


def _slots(kind, tokens, blocks, rng):
    if kind == "runs":  # runs of random lengths from random places
        ids, out, b = rng.permutation(blocks), [], 0
        while len(out) < tokens:
            n, o = min(int(rng.integers(1, 50)), tokens - len(out)), int(rng.integers(0, 16))
            out += [int(ids[b + (o + i) // 16]) * 16 + (o + i) % 16 for i in range(n)]
            b += (o + n - 1) // 16 + 1
        out = np.array(out)
    elif kind == "prompt":
        out = np.zeros(tokens)
    elif kind == "backwards":  # successive slots, falling
        out = 16 * (blocks - 1) + 7 - np.arange(tokens)
    else:
        out = rng.permutation(blocks * 16)[:tokens]
    out = out.astype(np.int64)
    if kind == "prompt":  # one run from an odd place, and padding
        out = 16 * 3 + 11 + np.arange(tokens)
        out[-2:] = -1
        return out
    if tokens > 3:
        out[rng.random(tokens) < 0.1] = -1
        out[-1] = -2 ** 31
    return out


def _run(dtype, kv, layout, tokens, hk, dk, hv, dv, kind, strided, special=False, seed=0, extra_bad=False):
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    blocks = tokens + 4
    elem = 1 if kv else TORCH[dtype].itemsize
    ks, vs = cache_shapes(blocks, hk, dk, hv, dv, layout, elem)
    cdt = torch.uint8 if kv else TORCH[dtype]
    kc0 = torch.randint(0, 256, ks + (cdt.itemsize,), generator=gen, dtype=torch.uint8).view(cdt).squeeze(-1).contiguous()
    vc0 = torch.randint(0, 256, vs + (cdt.itemsize,), generator=gen, dtype=torch.uint8).view(cdt).squeeze(-1).contiguous()
    if strided:
        row = torch.randn((tokens, 64 + hk * dk + hv * dv), generator=gen).to(TORCH[dtype])
        key, value = row[:, 64:64 + hk * dk].unflatten(1, (hk, dk)), row[:, 64 + hk * dk:].unflatten(1, (hv, dv))
    else:  # head-major rows
        key = torch.randn((hk, tokens, dk), generator=gen).to(TORCH[dtype]).transpose(0, 1)
        value = torch.randn((tokens, hv, dv), generator=gen).to(TORCH[dtype])
    if special:
        for x in (key, value):
            x[0, 0, :12] = torch.tensor([float("nan"), float("inf"), float("-inf"), 6e4, -6e4, 460.0, 448.0, 449.0, 1e-7,
                                         -0.0, 2.0 ** -10, 3 * 2.0 ** -11])
    slots = _slots(kind, tokens, blocks, rng)
    if extra_bad:
        slots[1], slots[2] = blocks * 16, 2 ** 31 - 1
    k_scale, v_scale = (0.37, 1.9) if kv and not special else (1.0, 1.0)
    kc, vc = kc0.to(DEV), vc0.to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    big = torch.empty((tokens, 64 + hk * dk + hv * dv), dtype=TORCH[dtype], device=DEV)
    if strided:  # the same strides on the GPU
        big.copy_(row if not special else torch.cat([row[:, :64], key.flatten(1), value.flatten(1)], 1))
        dkey, dvalue = big[:, 64:64 + hk * dk].unflatten(1, (hk, dk)), big[:, 64 + hk * dk:].unflatten(1, (hv, dv))
    else:
        dkey, dvalue = key.transpose(0, 1).contiguous().to(DEV).transpose(0, 1), value.to(DEV)
    pa.pa_append_kv(dkey, dvalue, kc, vc, _int(slots), layout=layout, kv_dtype=kv, k_scale=k_scale, v_scale=v_scale,
                    dev_error=err)
    torch.cuda.synchronize()
    assert int(err) == (pa.PA_DEVERR_SLOT if extra_bad else 0)
    for name, x, c0, c, is_key, scale in (("key", key, kc0, kc, True, k_scale), ("value", value, vc0, vc, False, v_scale)):
        want = store_ref(c0.view(BITS[elem]).numpy(), _quantised(x.contiguous(), kv, scale), slots, layout, is_key)
        got = c.cpu().view(BITS[elem]).numpy()
        if special and kv:  # any NaN is as good as another
            nan = lambda a: torch.isnan(torch.from_numpy(a).view(FP8[kv]).float()).numpy()  # noqa: E731
            assert np.array_equal(nan(got), nan(want))
            got, want = np.where(nan(got), 0, got), np.where(nan(want), 0, want)
        assert np.array_equal(got, want), (name, np.argwhere(got != want)[:4], int((got != want).sum()))


@pytest.mark.parametrize("layout", ["split", "nhd"])
@pytest.mark.parametrize("dtype,kv", TYPES)
@pytest.mark.parametrize("tokens,kind", [(1, "random"), (2, "runs"), (31, "runs"), (32, "runs"), (33, "random"),
                                         (100, "runs"), (70, "backwards")])
def test_append(dtype, kv, layout, tokens, kind):
    _run(dtype, kv, layout, tokens, 2, 64, 2, 64, kind, strided=tokens % 2 == 0, seed=tokens)


@pytest.mark.parametrize("layout", ["split", "nhd"])
@pytest.mark.parametrize("dtype,kv", TYPES)
@pytest.mark.parametrize("hk,dk,hv,dv", [(1, 128, 1, 128), (2, 64, 1, 128), (6, 128, 3, 256), (4, 256, 5, 64)])
def test_append_heads_and_sizes(dtype, kv, layout, hk, dk, hv, dv):
    _run(dtype, kv, layout, 83, hk, dk, hv, dv, "runs", strided=True, seed=hk + dv)


@pytest.mark.parametrize("layout", ["split", "nhd"])
@pytest.mark.parametrize("dtype,kv", TYPES)
@pytest.mark.parametrize("kind,tokens,hk,hv,size", [("prompt", 3001, 2, 2, 128), ("runs", 2700, 1, 2, 64),
                                                    ("random", 1500, 2, 2, 256), ("prompt", 2432, 1, 1, 256)])
def test_append_many_rows(dtype, kv, layout, kind, tokens, hk, hv, size):
    """Blocks of 32 rows and more, which begin with a page where they can."""
    _run(dtype, kv, layout, tokens, hk, size, hv, size, kind, strided=True, seed=tokens)


@pytest.mark.parametrize("layout", ["split", "nhd"])
@pytest.mark.parametrize("dtype,kv", TYPES)
def test_append_special_values_and_slots_past_the_cache(dtype, kv, layout):
    _run(dtype, kv, layout, 40, 2, 64, 2, 64, "runs", strided=True, special=True, seed=3)
    _run(dtype, kv, layout, 40, 2, 64, 2, 64, "random", strided=False, seed=4, extra_bad=True)


@pytest.mark.parametrize("layout", ["split", "nhd"])
def test_append_past_32_bits(layout):
    """Pages whose byte offset passes 2^32: the last ones of caches of 2.2e9 elements."""
    blocks, h, d = 135000, 8, 128
    ks, vs = cache_shapes(blocks, h, d, h, d, layout, 2)
    kc, vc = torch.zeros(ks, dtype=torch.float16, device=DEV), torch.zeros(vs, dtype=torch.float16, device=DEV)
    key, value = torch.randn((40, h, d), device=DEV).half(), torch.randn((40, h, d), device=DEV).half()
    slots = np.concatenate([np.arange(20) + 16 * (blocks - 2) + 5, np.arange(20) + 3])
    pa.pa_append_kv(key, value, kc, vc, _int(slots), layout=layout)
    b, o = torch.from_numpy(slots // 16).to(DEV), torch.from_numpy(slots % 16).to(DEV)
    got_k = kc[b, :, o] if layout == "nhd" else kc[b, :, :, o].flatten(2)
    got_v = vc[b, :, o] if layout == "nhd" else vc[b, :, :, o]
    assert torch.equal(got_k, key) and torch.equal(got_v, value)
    assert int(torch.count_nonzero(kc)) == int(torch.count_nonzero(key))
    assert int(torch.count_nonzero(vc)) == int(torch.count_nonzero(value))


def test_append_graph_and_other_stream():
    key, value = torch.randn((50, 2, 64), device=DEV).half(), torch.randn((50, 2, 64), device=DEV).half()
    slots = _int(np.arange(50) + 9)
    ref = torch.zeros((8, 2, 16, 64), dtype=torch.float16, device=DEV)
    for t in range(50):
        ref[(t + 9) // 16, :, (t + 9) % 16] = value[t]
    kc, vc = torch.zeros_like(ref), torch.zeros_like(ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pa.pa_append_kv(key, value, kc, vc, slots, layout="nhd", stream=side)
    side.synchronize()
    assert torch.equal(vc, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_append_kv(key, value, kc, vc, slots, layout="nhd")
    vc.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(vc, ref)
