"""The operators of a serving step together, as they are used: pages handed out
(pa_build_tables), the step's keys and values stored (pa_append_kv), attention over
the cache (pa_decode, or pa_diff_decode on a differential cache), step after step in
place.  The reference keeps every sequence's keys and values in plain lists of 64-bit
rows (fp8 caches: of the values they stand for) and attends over those, so a page in
the wrong place, a token lost or a length off by one shows.
"""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import paged_kv_attention_v2_gb300 as pa  # noqa: E402
from cache_ref import cache_shapes  # noqa: E402

DEV = "cuda:0"
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
# half a step of the output relative to itself, plus what the softmax weights (half
# a step of 16 bits in all but fp32) and the sums of a few hundred terms add to a
# convex combination of values of magnitude up to 5: 2^-11 x 5 and 2^-23 x 300 x 5
TOL = {"f16": (3e-3, 2.0 ** -11), "bf16": (3e-3, 2.0 ** -8), "f32": (2e-4, 2.0 ** -22)}


class Model:
    """One layer's cache and its plain counterpart."""

    def __init__(self, seed, n, dtype, kv, layout, diff, rows, max_len=400, kv_heads=2, group=2, size=64):
        self.n, self.dtype, self.kv, self.layout, self.diff, self.rows = n, dtype, kv, layout, diff, rows
        self.kv_heads, self.heads, self.size, self.max_len = kv_heads, kv_heads * group, size, max_len
        self.kh, self.vs = (2 * kv_heads, 2 * size) if diff else (kv_heads, size)
        width, self.rng = -(-max_len // 16), np.random.default_rng(seed)
        self.gen = torch.Generator().manual_seed(seed)
        blocks = n * width
        ct = FP8[kv] if kv else TORCH[dtype]
        ks, vs = cache_shapes(blocks, self.kh, size, kv_heads, self.vs, layout, ct.itemsize)
        nan = lambda s: torch.full(s, float("nan"), device=DEV).to(ct)  # noqa: E731  (a slot never stored shows)
        self.kc, self.vc = nan(ks), nan(vs)
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)  # noqa: E731
        self.i32 = i32
        self.table, self.lens = i32(np.full((n, width), -1)), i32(np.zeros(n))
        self.ring, self.pool = i32(self.rng.permutation(blocks)), i32([0, blocks])
        self.counter, self.err = i32([0]), i32([0])
        self.slots, self.positions = i32(np.zeros(rows)), i32(np.zeros(rows))
        self.start, self.keep = i32(np.zeros(n + 1)), i32(np.zeros(n))
        td = TORCH[dtype]
        row = torch.zeros((rows, self.kh * size + kv_heads * self.vs), dtype=td, device=DEV)  # as a projection leaves them
        self.row = row
        self.key = row[:, :self.kh * size].unflatten(1, (self.kh, size))
        self.value = row[:, self.kh * size:].unflatten(1, (kv_heads, self.vs))
        q = (rows, self.heads, 2, size) if diff else (rows, self.heads, size)
        self.query = torch.zeros(q, dtype=td, device=DEV)
        self.out = torch.zeros((rows, self.heads, self.vs), dtype=td, device=DEV)
        self.lam = torch.rand(self.heads, generator=self.gen).to(DEV) if diff else None
        self.scale_k, self.scale_v = (0.031, 0.027) if kv else (1.0, 1.0)
        self.most = 4
        if diff:
            self.ws = pa.alloc_diff_workspace(rows, self.heads, size, max_len, DEV)
        else:
            self.ws = pa.alloc_workspace(n, self.heads, size, max_len, DEV, num_query_tokens=rows)
        self.k_rows = [[] for _ in range(n)]
        self.v_rows = [[] for _ in range(n)]

    def step(self):
        """One step on the GPU: three calls, nothing read back."""
        pa.pa_build_tables(self.table, self.lens, self.ring, self.pool, self.slots, max_seq_len=self.max_len,
                           keep_lens=self.keep, query_start=self.start, positions=self.positions,
                           done_counter=self.counter, dev_error=self.err)
        pa.pa_append_kv(self.key, self.value, self.kc, self.vc, self.slots, layout=self.layout, kv_dtype=self.kv,
                        k_scale=self.scale_k, v_scale=self.scale_v, dev_error=self.err)
        kw = dict(num_kv_heads=self.kv_heads, scale=self.size ** -0.5, max_seq_len=self.max_len, layout=self.layout,
                  kv_dtype=self.kv, k_scale=self.scale_k, v_scale=self.scale_v, query_start=self.start,
                  max_query_len=self.most, dev_error=self.err, **self.ws)
        if self.diff:
            pa.pa_diff_decode(self.out, self.query, self.kc, self.vc, self.table, self.lens, lambdas=self.lam, norm=False,
                              **kw)
        else:
            kc, vc = (self.kc.view(torch.uint8), self.vc.view(torch.uint8)) if self.kv else (self.kc, self.vc)
            pa.pa_decode(self.out, self.query, kc, vc, self.table, self.lens, **kw)

    def inputs(self, keep, new):
        """This step's inputs, copied into the buffers that the calls use."""
        start = np.concatenate([[0], np.cumsum(new)])
        self.keep_np, self.new_np, self.start_np = keep, new, start
        self.start.copy_(self.i32(start))
        self.keep.copy_(self.i32(keep))
        self.row.copy_(torch.randn(self.row.shape, generator=self.gen).to(self.row.dtype).to(DEV))
        self.query.copy_(torch.randn(self.query.shape, generator=self.gen).to(self.query.dtype).to(DEV))
        self.out.fill_(7.0)

    def stored(self, x, scale):
        if self.kv is None:
            return x.double().cpu().numpy()
        top = torch.finfo(FP8[self.kv]).max
        q = (x.float() * (torch.tensor(1.0) / torch.tensor(scale)).item()).clamp(-top, top).to(FP8[self.kv])
        return q.double().cpu().numpy() * np.float32(scale)

    def check(self):
        torch.cuda.synchronize()
        assert int(self.err) == 0
        k, v, q = self.stored(self.key, self.scale_k), self.stored(self.value, self.scale_v), self.query.double().cpu().numpy()
        got = self.out.double().cpu().numpy()
        lens, positions, slots = self.lens.cpu().numpy(), self.positions.cpu().numpy(), self.slots.cpu().numpy()
        abs_tol, rel = TOL[self.dtype]
        lam = None if self.lam is None else self.lam.double().cpu().numpy()
        for s in range(self.n):
            del self.k_rows[s][self.keep_np[s]:], self.v_rows[s][self.keep_np[s]:]
            first = self.start_np[s]
            for t in range(first, self.start_np[s + 1]):
                assert positions[t] == len(self.k_rows[s])
                self.k_rows[s].append(k[t])
                self.v_rows[s].append(v[t])
            assert lens[s] == len(self.k_rows[s])
            for i, t in enumerate(range(first, self.start_np[s + 1])):
                seen = self.keep_np[s] + i + 1
                ks, vs = np.array(self.k_rows[s][:seen]), np.array(self.v_rows[s][:seen])
                for h in range(self.heads):
                    g = h // (self.heads // self.kv_heads)

                    def one(query, keys):
                        z = self.size ** -0.5 * keys @ query
                        p = np.exp(z - z.max())
                        return (p / p.sum()) @ vs[:, g]
                    if self.diff:
                        want = one(q[t, h, 0], ks[:, 2 * g]) - lam[h] * one(q[t, h, 1], ks[:, 2 * g + 1])
                    else:
                        want = one(q[t, h], ks[:, g])
                    assert np.all(np.abs(got[t, h] - want) <= 2 * abs_tol + rel * np.abs(want)), (s, i, h)
        last = self.start_np[-1]
        assert np.all(slots[last:] == -1) and np.all(got[last:] == 7.0)  # padding: no slot, rows left as they were


def _plan(m, step):
    """Prompts, growth, rejected drafts, an end and a new prompt."""
    held = np.array([len(r) for r in m.k_rows])
    keep = held.copy()
    new = m.rng.integers(0, m.most + 1, m.n)
    if step % 3 == 2:
        keep = np.maximum(held - m.rng.integers(0, 4, m.n), 0)
    if step % 4 == 3:
        keep[step % m.n], new[step % m.n] = 0, m.most if step % 8 == 3 else 0
    return keep, np.minimum(new, m.max_len - keep)


CASES = [("f16", None, "split", False), ("bf16", "e4m3", "nhd", False), ("f16", None, "nhd", True), ("bf16", "e5m2", "split", True),
         ("f32", None, "split", True)]


@pytest.mark.parametrize("dtype,kv,layout,diff", CASES)
def test_steps(dtype, kv, layout, diff):
    m = Model(3, 5, dtype, kv, layout, diff, rows=26)
    for step in range(14):
        m.inputs(*_plan(m, step))
        m.step()
        m.check()


@pytest.mark.parametrize("dtype,kv,layout,diff", CASES)
def test_steps_of_one_graph(dtype, kv, layout, diff):
    """One captured step replayed over changing lengths, offsets and inputs."""
    m = Model(4, 4, dtype, kv, layout, diff, rows=20)
    m.inputs(*_plan(m, 0))
    m.step()
    m.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.step()
    for step in range(1, 12):
        m.inputs(*_plan(m, step))
        g.replay()
        m.check()


def test_prompt_through_the_pages_then_decode():
    """A prompt stored over several calls (more tokens than one decode call attends
    with), then single tokens."""
    m = Model(5, 3, "bf16", None, "split", True, rows=330)
    m.most = 1
    for keep, new in ((np.zeros(3, dtype=int), np.array([100, 33, 197])), (np.array([100, 33, 197]), np.array([90, 160, 80]))):
        m.inputs(keep, new)
        pa.pa_build_tables(m.table, m.lens, m.ring, m.pool, m.slots, max_seq_len=m.max_len, keep_lens=m.keep,
                           query_start=m.start, done_counter=m.counter, dev_error=m.err)
        pa.pa_append_kv(m.key, m.value, m.kc, m.vc, m.slots, dev_error=m.err)
        k, v = m.key.double().cpu().numpy(), m.value.double().cpu().numpy()
        for s in range(3):
            m.k_rows[s] += list(k[m.start_np[s]:m.start_np[s + 1]])
            m.v_rows[s] += list(v[m.start_np[s]:m.start_np[s + 1]])
    for _ in range(3):
        m.inputs(np.array([len(r) for r in m.k_rows]), np.ones(3, dtype=int))
        m.step()
        m.check()


def test_two_streams_with_pools_of_their_own():
    """Two layers' steps on two streams at once, each with its own state."""
    a, b = Model(6, 5, "f16", None, "split", False, rows=26), Model(7, 5, "bf16", "e4m3", "nhd", True, rows=26)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for step in range(5):
        for m in (a, b):
            m.inputs(*_plan(m, step))
        torch.cuda.synchronize()
        for m, s in ((a, sa), (b, sb)):
            with torch.cuda.stream(s):
                m.step()
        a.check()
        b.check()
