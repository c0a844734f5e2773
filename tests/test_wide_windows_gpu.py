"""GPU tests: a sliding window that reaches over any length is none, for sequences shorter than their query tokens
too (positions below zero minus a window of nearly 2^31)."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import paged_kv_attention_v2_gb300 as pa  # noqa: E402

DEV = "cuda:0"
# lengths below, at and above the call's 8 tokens per sequence
LENS, MOST = [0, 1, 3, 5, 8, 30, 700, 1300], 8


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _inputs(kv, layout, size, diff=False, seed=0):
    rng, gen = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    n, kv_heads, group = len(LENS), 2, 1 if diff else 2
    width = -(-max(LENS) // 16)
    blocks = n * width
    if kv == "e2m1":
        k, v = (torch.randint(0, 256, (blocks, kv_heads, 9 * size), generator=gen, dtype=torch.uint8) for _ in range(2))
        for c in (k, v):
            c[:, :, 8 * size:] = 0x28  # scales of 1/4
    else:
        k = torch.randn((blocks, kv_heads * (2 if diff else 1), 16, size), generator=gen).half()
        v = torch.randn((blocks, kv_heads, 16, size * (2 if diff else 1)), generator=gen).half()
        if layout == "split":
            k, v = k.unflatten(3, (size // 8, 8)).permute(0, 1, 3, 2, 4).contiguous(), v.transpose(2, 3).contiguous()
    rows, heads = n * MOST, kv_heads * group
    q = torch.randn((rows, heads, 2, size) if diff else (rows, heads, size), generator=gen).half()
    table = rng.permutation(blocks).reshape(n, width)
    kw = dict(num_kv_heads=kv_heads, scale=size ** -0.5, max_seq_len=max(LENS), layout=layout, kv_dtype=kv,
              query_start=_int(np.arange(n + 1) * MOST), max_query_len=MOST)
    return q.to(DEV), k.to(DEV), v.to(DEV), _int(table), _int(LENS), heads, kw


WIDE = [2 ** 31 - 2, 2 ** 31 - 5, 2 ** 31 - 14, 1300]


@pytest.mark.parametrize("mode", ["v1", "v2", "v2f"])
@pytest.mark.parametrize("kv,layout,size", [(None, "split", 64), (None, "nhd", 128), ("e2m1", "nhd", 64), ("e2m1", "nhd", 128)])
def test_decode(kv, layout, size, mode):
    q, k, v, table, lens, heads, kw = _inputs(kv, layout, size)
    results = []
    for window in [-1] + WIDE:
        ws = pa.alloc_workspace(len(LENS), heads, size, max(LENS), DEV, num_query_tokens=q.shape[0], num_kv_heads=2 if mode == "v2f" else None)
        for name in ("exp_sums", "max_logits", "tmp_out"):
            ws[name].fill_(float("nan"))
        out, err = torch.full_like(q, 7.0), _int([0])
        pa.pa_decode(out, q, k, v, table, lens, mode=mode[:2], window_left=window, dev_error=err, **kw, **ws)
        torch.cuda.synchronize()
        assert int(err) == 0
        results.append((out, ws["exp_sums"], ws["max_logits"]))
    assert torch.isfinite(results[0][0]).all()
    for r in results[1:]:
        for a, b in zip(r, results[0]):
            assert torch.equal(a, b) or (mode == "v1" and a is not r[0])


@pytest.mark.parametrize("mode", ["v1", "v2"])
def test_diff_decode(mode):
    q, k, v, table, lens, heads, kw = _inputs(None, "nhd", 64, diff=True)
    lam = torch.rand(heads, device=DEV)
    results = []
    for window in [-1] + WIDE:
        ws = pa.alloc_diff_workspace(q.shape[0], heads, 64, max(LENS), DEV)
        out, err = torch.full((q.shape[0], heads, 128), 7.0, dtype=q.dtype, device=DEV), _int([0])
        pa.pa_diff_decode(out, q, k, v, table, lens, lambdas=lam, mode=mode, window_left=window, dev_error=err, **kw, **ws)
        torch.cuda.synchronize()
        assert int(err) == 0
        results.append(out)
    assert torch.isfinite(results[0]).all()
    assert all(torch.equal(r, results[0]) for r in results[1:])


@pytest.mark.parametrize("decay", [1.0, 0.5])
@pytest.mark.parametrize("kv,layout,size", [(None, "split", 64), ("e2m1", "nhd", 128)])
def test_weights(kv, layout, size, decay):
    q, k, v, table, lens, heads, kw = _inputs(kv, layout, size)
    ws = pa.alloc_workspace(len(LENS), heads, size, max(LENS), DEV, num_query_tokens=q.shape[0])
    pa.pa_decode(torch.empty_like(q), q, k, v, table, lens, mode="v2", **kw, **ws)
    results = []
    for window in [-1] + WIDE:
        scores, err = torch.full((k.shape[0], 2, 16), 0.25, device=DEV), _int([0])
        pa.pa_add_weights(scores, q, k, table, lens, ws["exp_sums"], ws["max_logits"], decay=decay, window_left=window, dev_error=err, **kw)
        torch.cuda.synchronize()
        assert int(err) == 0
        results.append(scores)
    assert all(torch.equal(r, results[0]) for r in results[1:])
    # every query token that sees a key has weights of one in all, of two heads to a kv head; what was there fades, and
    # tokens of the call are set
    for s, n in enumerate(LENS):
        t = torch.arange(n, device=DEV)
        got = results[0][table[s].long()[t // 16], :, t % 16].double().sum(0)
        seen = min(n, MOST)
        old = 0.25 * decay * max(n - MOST, 0)
        assert torch.allclose(got, torch.full_like(got, 2.0 * seen + old), rtol=2e-4, atol=1e-6), (s, got)
