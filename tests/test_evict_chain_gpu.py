"""The operators of a cache that is short of room together, as they are used: pages handed
out, keys and values stored, attention (v2, for its statistics), its weights added to the scores,
the tokens within the budget selected and moved to the front, and the next step on what is left.
The reference keeps plain lists of rows per sequence and kv head, and drops from them what the
selection (checked against the scores that it had) dropped."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import paged_kv_attention_v2_gb300 as pa  # noqa: E402
from cache_ref import cache_shapes  # noqa: E402
from short_ref import select_ref, store4, values4  # noqa: E402

DEV = "cuda:0"
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
# as in test_serving_step_gpu: half a step of the output, and what weights of 16 bits and the sums add
TOL = {"f16": (3e-3, 2.0 ** -11), "bf16": (3e-3, 2.0 ** -8), "f32": (2e-4, 2.0 ** -22)}


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


class Served:
    def __init__(self, seed, n, dtype, kv, layout, budget, sink, recent, decay, rows=14, kv_heads=2, group=2, size=64, max_len=96):
        self.n, self.dtype, self.kv, self.layout, self.rows = n, dtype, kv, layout, rows
        self.budget, self.sink, self.recent, self.decay = budget, sink, recent, decay
        self.kv_heads, self.group, self.heads, self.size, self.max_len = kv_heads, group, kv_heads * group, size, max_len
        self.rng, self.gen = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        width = -(-max_len // 16)
        blocks = n * width
        if kv == "e2m1":
            self.kc, self.vc = (torch.full((blocks, kv_heads, 9 * size), 0x7f, dtype=torch.uint8, device=DEV) for _ in range(2))
        else:
            ct = FP8[kv] if kv else TORCH[dtype]
            self.kc, self.vc = (torch.full(s, float("nan"), device=DEV).to(ct)
                                for s in cache_shapes(blocks, kv_heads, size, kv_heads, size, layout, ct.itemsize))
        self.scale_k, self.scale_v = (1.0, 1.0) if kv is None else ((0.0019, 0.0023) if kv == "e2m1" else (0.031, 0.027))
        self.scores = torch.full((blocks, kv_heads, 16), float("nan"), device=DEV)
        self.table, self.lens = i32(np.full((n, width), -1)), i32(np.zeros(n))
        self.ring, self.pool = i32(self.rng.permutation(blocks)), i32([0, blocks])
        self.counter, self.err = i32([0]), i32([0])
        self.slots, self.start = i32(np.zeros(rows)), i32(np.zeros(n + 1))
        self.keep, self.budgets = i32(np.zeros(n)), i32(np.full(n, budget))
        self.kept = i32(np.full((n, kv_heads, budget), -1))
        td = TORCH[dtype]
        self.key = torch.zeros((rows, kv_heads, size), dtype=td, device=DEV)
        self.value, self.query = torch.zeros_like(self.key), torch.zeros((rows, self.heads, size), dtype=td, device=DEV)
        self.out = torch.zeros_like(self.query)
        self.before = torch.zeros_like(self.scores)  # the scores that the selection saw
        self.ws = pa.alloc_workspace(n, self.heads, size, max_len, DEV, num_query_tokens=rows)
        self.lists = [[([], []) for _ in range(kv_heads)] for _ in range(n)]
        self.old = [[np.zeros(0) for _ in range(kv_heads)] for _ in range(n)]

    def step(self):
        """One step on the GPU: six calls, nothing read back."""
        pa.pa_build_tables(self.table, self.lens, self.ring, self.pool, self.slots, max_seq_len=self.max_len, keep_lens=self.keep,
                           query_start=self.start, done_counter=self.counter, dev_error=self.err)
        cache = dict(layout=self.layout, kv_dtype=self.kv, dev_error=self.err)
        pa.pa_append_kv(self.key, self.value, self.kc, self.vc, self.slots, k_scale=self.scale_k, v_scale=self.scale_v, **cache)
        kw = dict(num_kv_heads=self.kv_heads, scale=self.size ** -0.5, max_seq_len=self.max_len, query_start=self.start,
                  max_query_len=4, k_scale=self.scale_k, **cache)
        kc, vc = (self.kc.view(torch.uint8), self.vc.view(torch.uint8)) if self.kv else (self.kc, self.vc)
        pa.pa_decode(self.out, self.query, kc, vc, self.table, self.lens, mode="v2", v_scale=self.scale_v, **kw, **self.ws)
        pa.pa_add_weights(self.scores, self.query, self.kc, self.table, self.lens, self.ws["exp_sums"], self.ws["max_logits"],
                          decay=self.decay, **kw)
        self.before.copy_(self.scores)
        pa.pa_select_tokens(self.kept, self.keep, self.scores, self.table, self.lens, self.budgets, max_seq_len=self.max_len,
                            sink=self.sink, recent=self.recent, dev_error=self.err)
        pa.pa_compact_kv(self.kc, self.vc, self.table, self.kept, self.keep, scores=self.scores, **cache)

    def inputs(self):
        new = self.rng.integers(0, 5, self.n)
        self.start_np = np.concatenate([[0], np.cumsum(new)])
        self.start.copy_(i32(self.start_np))
        for t in (self.key, self.value, self.query):
            t.copy_(torch.randn(t.shape, generator=self.gen).to(t.dtype).to(DEV))
        self.out.fill_(7.0)

    def stored(self, x, g):
        x = x.double().cpu().numpy()
        if self.kv is None:
            return x
        if self.kv == "e2m1":
            rows = x.shape[0]
            pages = store4(np.zeros((-(-rows // 16), self.kv_heads, 9 * self.size), dtype=np.uint8), x, np.arange(rows), g)
            return values4(pages, g).transpose(0, 2, 1, 3).reshape(-1, self.kv_heads, self.size)[:rows]
        top = torch.finfo(FP8[self.kv]).max
        q = (torch.from_numpy(x).float() / torch.tensor(g)).clamp(-top, top).to(FP8[self.kv])
        return q.double().numpy() * np.float32(g)

    def check(self):
        torch.cuda.synchronize()
        assert int(self.err) == 0
        k, v, q = self.stored(self.key, self.scale_k), self.stored(self.value, self.scale_v), self.query.double().cpu().numpy()
        got, table, lens = self.out.double().cpu().numpy(), self.table.cpu().numpy(), self.lens.cpu().numpy()
        before, after = self.before.cpu().numpy(), self.scores.double().cpu().numpy()
        kept, keep = self.kept.cpu().numpy(), self.keep.cpu().numpy()
        absolute, relative = TOL[self.dtype]
        want_kept, want_keep = select_ref(before, table, lens, [self.budget] * self.n, self.sink, self.recent, self.budget, -1)
        assert np.array_equal(keep, want_keep)
        for s in range(self.n):
            first, end = self.start_np[s], self.start_np[s + 1]
            for g in range(self.kv_heads):
                keys, values = self.lists[s][g]
                keys += list(k[first:end, g])
                values += list(v[first:end, g])
                n = len(keys)
                assert lens[s] == n
                ks, vs, added = np.array(keys), np.array(values), np.zeros(n)
                for t in range(first, end):
                    seen = n - (end - t) + 1
                    for h in range(g * self.group, (g + 1) * self.group):
                        z = self.size ** -0.5 * ks[:seen] @ q[t, h]
                        w = np.exp(z - z.max())
                        w /= w.sum()
                        added[:seen] += w
                        o = w @ vs[:seen]
                        assert np.all(np.abs(got[t, h] - o) <= 2 * absolute + relative * np.abs(o)), (s, t, h)
                old = np.concatenate([self.old[s][g], np.zeros(end - first)])
                want = np.where(np.arange(n) >= n - (end - first), added, np.float64(np.float32(self.decay)) * old + added)
                at = (table[s, np.arange(n) // 16], g, np.arange(n) % 16)
                # the levels are a decode's statistics: logits off by some 1e-4, and as much in each step's sum
                assert np.all(np.abs(before[at] - want) <= 1e-3 * want + 1e-12), (s, g)
                stay = kept[s, g, :keep[s]]
                assert np.array_equal(stay, want_kept[s, g, :keep[s]])
                self.lists[s][g] = ([keys[i] for i in stay], [values[i] for i in stay])
                self.old[s][g] = before[at].astype(np.float64)[stay]
                at = (table[s, np.arange(keep[s]) // 16], g, np.arange(keep[s]) % 16)
                assert np.array_equal(after[at], self.old[s][g])


CASES = [("f16", None, "split", 1.0), ("bf16", "e4m3", "nhd", 0.9), ("f16", "e2m1", "nhd", 1.0), ("bf16", "e2m1", "nhd", 0.95),
         ("f32", None, "nhd", 1.0), ("bf16", "e5m2", "split", 1.0)]


@pytest.mark.parametrize("dtype,kv,layout,decay", CASES)
def test_steps_within_a_budget(dtype, kv, layout, decay):
    m = Served(3, 3, dtype, kv, layout, budget=37, sink=2, recent=9, decay=decay)
    for _ in range(30):
        m.inputs()
        m.step()
        m.check()


@pytest.mark.parametrize("dtype,kv,layout,decay", CASES[:3])
def test_steps_of_one_graph(dtype, kv, layout, decay):
    m = Served(4, 3, dtype, kv, layout, budget=20, sink=0, recent=4, decay=decay)
    m.inputs()
    m.step()
    m.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.step()
    for _ in range(25):
        m.inputs()
        g.replay()
        m.check()


def test_two_streams_at_once():
    a = Served(5, 3, "f16", "e2m1", "nhd", budget=30, sink=1, recent=5, decay=1.0)
    b = Served(6, 3, "bf16", None, "split", budget=25, sink=1, recent=5, decay=0.9)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(12):
        for m in (a, b):
            m.inputs()
        torch.cuda.synchronize()
        for m, s in ((a, sa), (b, sb)):
            with torch.cuda.stream(s):
                m.step()
        a.check()
        b.check()
