"""Many steps of serving enqueued one behind the other, with nothing waited for in
between: prompts of tens of thousands of rows and then drafted tokens, some of them
rejected, some sequences ended and begun anew, through pa_build_tables on many CTAs
(lengths and pool in place), pa_append_kv in its large blocks and the attention kernels.
Each of them may become resident while the one before it still runs, and reads what that
one writes.  Tables, slots and lengths are checked bit for bit, and every output against
plain rows in 64 bits.
"""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import paged_kv_attention_v2_gb300 as pa  # noqa: E402
from cache_ref import cache_shapes, tables_ref  # noqa: E402

DEV = "cuda:0"
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
# half a step of the output relative to itself, plus what the softmax weights (half a
# step of 16 bits in all but fp32) and the sums of a few hundred terms add to a convex
# combination of values of magnitude up to 5.5 (two of them in a differential head)
TOL = {"f16": (6e-3, 2.0 ** -11), "bf16": (6e-3, 2.0 ** -8), "f32": (4e-4, 2.0 ** -22)}
N, MOST, TOP, HEADS, SIZE = 300, 4, 288, 8, 64


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _plans(rng, steps):
    """(keep, new) of each step: all prompts, then drafts with cuts, ends and new prompts."""
    lens, out = np.zeros(N, dtype=np.int64), []
    for step in range(steps):
        keep = lens.copy()
        if step == 0:
            new = rng.integers(1, TOP - 60, N)
        elif step % 5 == 4:  # a fifth of the sequences begin anew, with prompts
            again = rng.random(N) < 0.2
            keep[again] = 0
            new = np.where(again, rng.integers(100, TOP - 60, N), 1)
        else:
            keep = np.maximum(lens - rng.integers(0, 3, N), 0)
            new = rng.integers(0, MOST + 1, N)
        new = np.minimum(new, TOP - keep)
        lens = keep + new
        out.append((keep, new))
    return out


class Chain:
    def __init__(self, dtype, kv, layout, diff, mode, steps=9):
        self.dtype, self.kv, self.layout, self.diff, self.mode = dtype, kv, layout, diff, mode
        rng, gen = np.random.default_rng(1), torch.Generator(device=DEV).manual_seed(2)
        self.kh, self.vs = (2 * HEADS, 2 * SIZE) if diff else (HEADS, SIZE)
        self.width = -(-TOP // 16)
        self.blocks = N * self.width
        ct, td = FP8[kv] if kv else TORCH[dtype], TORCH[dtype]
        ks, vs = cache_shapes(self.blocks, self.kh, SIZE, HEADS, self.vs, layout, ct.itemsize)
        nan = lambda s: torch.full(s, float("nan"), device=DEV).to(ct)  # noqa: E731
        self.kc, self.vc = nan(ks), nan(vs)
        self.ring0, self.pool0 = rng.permutation(self.blocks), np.array([777, self.blocks])
        self.table, self.lens = _int(np.full((N, self.width), -1)), _int(np.zeros(N))
        self.ring, self.pool = _int(self.ring0), _int(self.pool0)
        self.counter, self.err = _int([0]), _int([0])
        self.lam = torch.rand(HEADS, generator=gen, device=DEV) if diff else None
        self.scale_k, self.scale_v = (0.031, 0.027) if kv else (1.0, 1.0)
        self.steps = []
        for i, (keep, new) in enumerate(_plans(rng, steps)):
            rows = int(new.sum()) + 5
            row = torch.randn((rows, self.kh * SIZE + HEADS * self.vs), generator=gen, device=DEV).to(td)
            q = torch.randn((rows, HEADS, 2, SIZE) if diff else (rows, HEADS, SIZE), generator=gen, device=DEV).to(td)
            start = np.concatenate([[0], np.cumsum(new)])
            attend = new.max() <= MOST
            ws = None
            if attend:
                ws = pa.alloc_diff_workspace(rows, HEADS, SIZE, TOP, DEV) if diff else \
                    pa.alloc_workspace(N, HEADS, SIZE, TOP, DEV, num_query_tokens=rows)
            self.steps.append(dict(keep=keep, new=new, start=start, rows=rows, attend=attend, ws=ws, q=q, dkeep=_int(keep),
                                   dstart=_int(start), key=row[:, :self.kh * SIZE].unflatten(1, (self.kh, SIZE)),
                                   value=row[:, self.kh * SIZE:].unflatten(1, (HEADS, self.vs)),
                                   slots=_int(np.full(rows, 7)), out=torch.full((rows, HEADS, self.vs), 7.0, device=DEV).to(td),
                                   table=torch.empty_like(self.table), lens=torch.empty_like(self.lens)))

    def run(self):
        for s in self.steps:
            pa.pa_build_tables(self.table, self.lens, self.ring, self.pool, s["slots"], max_seq_len=TOP, keep_lens=s["dkeep"],
                               query_start=s["dstart"], done_counter=self.counter, dev_error=self.err)
            pa.pa_append_kv(s["key"], s["value"], self.kc, self.vc, s["slots"], layout=self.layout, kv_dtype=self.kv,
                            k_scale=self.scale_k, v_scale=self.scale_v, dev_error=self.err)
            if not s["attend"]:
                continue
            kw = dict(num_kv_heads=HEADS, scale=SIZE ** -0.5, max_seq_len=TOP, layout=self.layout, kv_dtype=self.kv,
                      k_scale=self.scale_k, v_scale=self.scale_v, query_start=s["dstart"], max_query_len=MOST, mode=self.mode,
                      dev_error=self.err, **s["ws"])
            if self.diff:
                pa.pa_diff_decode(s["out"], s["q"], self.kc, self.vc, self.table, self.lens, lambdas=self.lam, norm=False, **kw)
            else:
                kc, vc = (self.kc.view(torch.uint8), self.vc.view(torch.uint8)) if self.kv else (self.kc, self.vc)
                pa.pa_decode(s["out"], s["q"], kc, vc, self.table, self.lens, **kw)

    def reset(self):
        self.table.fill_(-1)
        self.lens.zero_()
        self.ring.copy_(_int(self.ring0))
        self.pool.copy_(_int(self.pool0))
        for s in self.steps:
            s["slots"].fill_(7)
            s["out"].fill_(7.0)

    def stored(self, x, scale):
        if self.kv is None:
            return x.double()
        top = torch.finfo(FP8[self.kv]).max
        q = (x.float() / torch.tensor(scale, device=DEV)).clamp(-top, top).to(FP8[self.kv])
        return q.double() * float(np.float32(scale))

    def check(self):
        torch.cuda.synchronize()
        assert int(self.err) == 0
        table, ring, state = np.full((N, self.width), -1), self.ring0.copy(), self.pool0.copy()
        lens = np.zeros(N, dtype=np.int64)
        keys = torch.zeros((N, TOP, self.kh, SIZE), dtype=torch.float64, device=DEV)
        values = torch.zeros((N, TOP, HEADS, self.vs), dtype=torch.float64, device=DEV)
        at = torch.arange(TOP, device=DEV)
        absolute, relative = TOL[self.dtype]
        for i, s in enumerate(self.steps):
            table, ring, slots, positions, lens, state = tables_ref(table, lens, ring, state, s["rows"], s["keep"], s["start"])
            assert np.array_equal(s["slots"].cpu().numpy(), slots), i
            rows = int(s["start"][-1])
            owner = torch.from_numpy(np.repeat(np.arange(N), s["new"])).to(DEV)
            pos = torch.from_numpy(positions[:rows]).to(DEV)
            keys[owner, pos] = self.stored(s["key"][:rows], self.scale_k)
            values[owner, pos] = self.stored(s["value"][:rows], self.scale_v)
            assert (s["out"][rows:] == 7).all()
            if not s["attend"]:
                continue
            seen = (at[None] <= pos[:, None])[:, :, None]

            def one(q, k):
                z = torch.einsum("rhd,rthd->rth", q.double(), k[owner]) * SIZE ** -0.5
                return torch.softmax(z.masked_fill(~seen, float("-inf")), 1)
            if self.diff:
                w = one(s["q"][:rows, :, 0], keys[:, :, 0::2]) - self.lam.double()[None, None] * one(s["q"][:rows, :, 1], keys[:, :, 1::2])
            else:
                w = one(s["q"][:rows], keys)
            want = torch.einsum("rth,rthd->rhd", w, values[owner])
            off = (s["out"][:rows].double() - want).abs() - absolute - relative * want.abs()
            assert float(off.max()) <= 0, (i, float(off.max()), int((off > 0).sum()))
        assert np.array_equal(self.table.cpu().numpy(), table) and np.array_equal(self.lens.cpu().numpy(), lens)
        assert np.array_equal(self.ring.cpu().numpy(), ring) and np.array_equal(self.pool.cpu().numpy(), state)


CASES = [("f16", None, "split", False, "v2"), ("bf16", "e4m3", "nhd", False, "v1"), ("f16", None, "nhd", True, "v1"),
         ("bf16", "e4m3", "split", True, "v2"), ("f32", None, "split", True, "auto")]


@pytest.mark.parametrize("dtype,kv,layout,diff,mode", CASES)
def test_steps_without_a_wait_between(dtype, kv, layout, diff, mode):
    c = Chain(dtype, kv, layout, diff, mode)
    torch.cuda.synchronize()
    for _ in range(3):
        c.run()
        c.check()
        c.reset()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    g.replay()
    c.check()
