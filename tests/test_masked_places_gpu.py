"""GPU tests: keys and values that no query token sees (before the sliding window, in the page that the window begins in and
the one before; behind the end) reach neither a decode over 4-bit pages nor the attention weights, where they are NaN or
infinite: outputs and scores against the formula in 64 bits over the seen tokens."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import paged_kv_attention_v2_gb300 as pa  # noqa: E402
from short_ref import attention, pages4, row_weights, sequences, store4, values4  # noqa: E402

DEV = "cuda:0"
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
# as in test_fp4_gpu and test_evict_gpu
TOL = {"f16": (6e-3, 2.0 ** -11), "bf16": (6e-3, 2.0 ** -8)}
REL = 2e-4


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _batch(rng, lens):
    own = [-(-x // 16) for x in lens]
    ids = rng.permutation(sum(own))
    table = np.zeros((len(lens), max(own)), dtype=np.int64)
    at = np.concatenate([[0], np.cumsum(own)])
    for s in range(len(lens)):
        table[s, :own[s]] = ids[at[s]:at[s + 1]]
    return table, len(ids)


def _unseen(lens, q_len, window):
    """(sequence, token) of places that no row sees: before the first row's window, and behind the end."""
    out = []
    for s, n in enumerate(lens):
        qn = q_len[s] if q_len else 1
        first = max(0, n - qn - window)
        out += [(s, t) for t in (first - 1, first - 2, first - 7, first - 16, first - 17) if t >= 0]
        out += [(s, t) for t in range(n, -(-n // 16) * 16)]
    return out


def _four_bits(rng, gen, table, blocks, kv_heads, size, odd, g):
    """A 4-bit cache whose block scales are NaN at `odd`, and what it stands for."""
    flat = torch.randn((blocks * 16, kv_heads, size), generator=gen).half().double().numpy()
    c = store4(pages4(blocks, kv_heads, size), flat, np.arange(blocks * 16), g)
    for s, t in odd:
        at = 8 * size + (t % 16) * (size // 16)
        c[table[s, t // 16], :, at:at + size // 16] = rng.choice([0x7f, 0xff])
    return c, values4(c, g)


LENS = [5, 40, 700, 1037]
SEVERAL = [None, [2, 4, 1, 3]]


@pytest.mark.parametrize("mode", ["v1", "v2"])
@pytest.mark.parametrize("q_len", SEVERAL)
@pytest.mark.parametrize("dtype,size,group", [("f16", 64, 2), ("bf16", 128, 3), ("f16", 128, 4), ("bf16", 64, 1)])
def test_decode_over_4_bit_pages(dtype, size, group, q_len, mode):
    for window in (0, 3, 100, 600):
        rng, gen = np.random.default_rng(window), torch.Generator().manual_seed(window)
        kv_heads, ks, vs = 2, 0.0019, 0.0023
        table, blocks = _batch(rng, LENS)
        odd = _unseen(LENS, q_len, window)
        (kc, k), (vc, v) = (_four_bits(rng, gen, table, blocks, kv_heads, size, odd, g) for g in (ks, vs))
        rows = sum(q_len) if q_len else len(LENS)
        start = np.concatenate([[0], np.cumsum(q_len)]) if q_len else np.arange(len(LENS) + 1)
        q = torch.randn((rows, kv_heads * group, size), generator=gen).to(TORCH[dtype])
        out, err = torch.full(q.shape, 7.0, dtype=TORCH[dtype], device=DEV), _int([0])
        ws = pa.alloc_workspace(len(LENS), kv_heads * group, size, max(LENS), DEV, num_query_tokens=rows)
        kw = dict(query_start=_int(start), max_query_len=4) if q_len else {}
        pa.pa_decode(out, q.to(DEV), torch.from_numpy(kc).to(DEV), torch.from_numpy(vc).to(DEV), _int(table), _int(LENS), mode=mode,
                     num_kv_heads=kv_heads, scale=size ** -0.5, max_seq_len=max(LENS), layout="nhd", kv_dtype="e2m1", k_scale=ks,
                     v_scale=vs, window_left=window, dev_error=err, **kw, **ws)
        torch.cuda.synchronize()
        assert int(err) == 0
        want = attention(q.double().numpy(), sequences(k, table, LENS), sequences(v, table, LENS), LENS, start, group,
                         size ** -0.5, window=window)
        got = out.double().cpu().numpy()
        absolute, relative = TOL[dtype]
        assert np.all(np.abs(got - want) <= absolute + relative * np.abs(want)), window


KINDS = [("f32", None, "nhd"), ("f16", None, "split"), ("bf16", None, "nhd"), ("bf16", "e4m3", "split"), ("f16", "e4m3", "nhd"),
         ("f16", "e5m2", "split"), ("bf16", "e5m2", "nhd"), ("f16", "e2m1", "nhd"), ("bf16", "e2m1", "nhd")]


@pytest.mark.parametrize("q_len", SEVERAL)
@pytest.mark.parametrize("size,group", [(64, 1), (128, 3), (64, 4)])
@pytest.mark.parametrize("dtype,kv,layout", KINDS)
def test_weights(dtype, kv, layout, size, group, q_len):
    for window, decay in ((0, 1.0), (3, 0.0), (100, 0.9), (600, 1.0)):
        rng, gen = np.random.default_rng(window), torch.Generator().manual_seed(window)
        kv_heads, heads = 2, 2 * group
        table, blocks = _batch(rng, LENS)
        odd = _unseen(LENS, q_len, window)
        if kv == "e2m1":
            ks = 0.0019
            c, values = _four_bits(rng, gen, table, blocks, kv_heads, size, odd, ks)
            cache = torch.from_numpy(c).to(DEV)
        else:
            ks = 2.0 ** -5 if kv else 1.0
            x = torch.randn((blocks, kv_heads, 16, size), generator=gen) / ks
            for i, (s, t) in enumerate(odd):
                x[table[s, t // 16], :, t % 16, (37 * i) % size] = float("nan") if kv == "e4m3" or i % 2 else float("inf")
            c = x.to(FP8[kv] if kv else TORCH[dtype])
            values = c.double().numpy() * ks
            if layout == "split":
                w = 16 // c.element_size()
                c = c.unflatten(3, (size // w, w)).permute(0, 1, 3, 2, 4)
            cache = c.contiguous().to(DEV)
        rows = sum(q_len) if q_len else len(LENS)
        start = np.concatenate([[0], np.cumsum(q_len)]) if q_len else np.arange(len(LENS) + 1)
        q = torch.randn((rows, heads, size), generator=gen).to(TORCH[dtype])
        parts = -(-max(LENS) // 512)
        most, sums = np.full((rows, heads, parts), -np.inf), np.zeros((rows, heads, parts))
        scores = rng.random((blocks, kv_heads, 16)).astype(np.float32)
        want = scores.astype(np.float64)
        for s, n in enumerate(LENS):
            k, qn = sequences(values, table, LENS)[s], int(start[s + 1] - start[s])
            added = np.zeros((n, kv_heads))
            for r in range(start[s], start[s + 1]):
                pos = n - (int(start[s + 1]) - r)
                lo = max(0, pos - window)
                for h in range(heads):
                    z = size ** -0.5 * k[lo:pos + 1, h // group] @ q[r, h].double().numpy()
                    for p in range(lo // 512, pos // 512 + 1):
                        zp = z[max(p * 512 - lo, 0):(p + 1) * 512 - lo]
                        most[r, h, p] = np.float32(zp.max())
                        sums[r, h, p] = np.exp(zp - most[r, h, p]).sum()
                    added[lo:pos + 1, h // group] += row_weights(q[r, h].double().numpy(), k[:, h // group], size ** -0.5, lo, pos)
            t = np.arange(n)
            at = (table[s, t // 16], slice(None), t % 16)
            old = np.where((t < n - qn)[:, None], float(np.float32(decay)) * want[at], 0.0)
            want[at] = old + added
        got, err = torch.from_numpy(scores).to(DEV), _int([0])
        kw = dict(query_start=_int(start), max_query_len=4) if q_len else {}
        pa.pa_add_weights(got, q.to(DEV), cache, _int(table), _int(LENS), torch.from_numpy(sums.astype(np.float32)).to(DEV),
                          torch.from_numpy(most.astype(np.float32)).to(DEV), num_kv_heads=kv_heads, scale=size ** -0.5,
                          max_seq_len=max(LENS), decay=decay, layout=layout, window_left=window, kv_dtype=kv, k_scale=ks, dev_error=err, **kw)
        torch.cuda.synchronize()
        assert int(err) == 0
        out = got.double().cpu().numpy()
        ok = np.abs(out - want) <= REL * np.abs(want) + 1e-30
        assert ok.all(), (window, decay, np.argwhere(~ok)[:4], out[~ok][:4], want[~ok][:4])
