"""GPU tests of pa_decode and pa_diff_decode: tokens before the sliding window do not
reach the output, even where their keys or values are infinite or NaN.  (Slots behind
the end are NaN in the other tests of these calls.)  Every output against the formula in
64 bits over the seen tokens.
"""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import paged_kv_attention_v2_gb300 as pa  # noqa: E402

DEV = "cuda:0"
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPES = [("f32", None), ("f16", None), ("bf16", None), ("f16", "e4m3"), ("bf16", "e5m2"), ("bf16", "e4m3"), ("f16", "e5m2")]
# half a step of the output, plus half a step of 16 bits of the weights of values up to
# 5 (two maps of them), and what 2e-5 of the logits' sums (fp32: 4e-6) makes of those
TOL = {"f16": (6e-3, 2.0 ** -11), "bf16": (6e-3, 2.0 ** -8), "f32": (4e-4, 2.0 ** -22)}


def _cache(rows, ct, layout, is_key):
    c = rows.to(ct)
    x = 16 // ct.itemsize
    if layout == "split":
        c = c.unflatten(3, (rows.shape[3] // x, x)).permute(0, 1, 3, 2, 4) if is_key else c.transpose(2, 3)
    return c.contiguous().to(DEV)


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _run(diff, dtype, kv, layout, size, kv_heads, group, lens, q_len, window, odd, mode, seed=0):
    """odd: (sequence, token, in the keys?, value) of each place that is no number."""
    rng, gen = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    n, heads = len(lens), kv_heads * group
    kh, vs = (2 * kv_heads, 2 * size) if diff else (kv_heads, size)
    own = [-(-x // 16) for x in lens]
    ids = rng.permutation(sum(own))
    table = np.zeros((n, max(own)), dtype=np.int64)
    at = np.concatenate([[0], np.cumsum(own)])
    for s in range(n):
        table[s, :own[s]] = ids[at[s]:at[s + 1]]
    ct = FP8[kv] if kv else TORCH[dtype]
    k = torch.randn((len(ids), kh, 16, size), generator=gen)
    v = torch.randn((len(ids), kv_heads, 16, vs), generator=gen)
    for i, (s, t, key, value) in enumerate(odd):
        x, h = (k, (3 * i) % kh) if key else (v, i % kv_heads)
        x[table[s, t // 16], h, t % 16, (37 * i + 5) % x.shape[3]] = value
    kc, vc = _cache(k, ct, layout, True), _cache(v, ct, layout, False)
    k, v = k.to(ct).double().numpy(), v.to(ct).double().numpy()
    rows = sum(q_len) if q_len else n
    start = np.concatenate([[0], np.cumsum(q_len)]) if q_len else np.arange(n + 1)
    q = torch.randn((rows, heads, 2, size) if diff else (rows, heads, size), generator=gen).to(TORCH[dtype])
    lam = torch.rand(heads, generator=gen)
    out = torch.full((rows, heads, vs), 7.0, dtype=TORCH[dtype], device=DEV)
    top = max(lens)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw = dict(num_kv_heads=kv_heads, scale=size ** -0.5, max_seq_len=top, layout=layout, kv_dtype=kv, window_left=window,
              mode=mode, dev_error=err)
    if q_len:
        kw.update(query_start=_int(start), max_query_len=max(q_len))
    if diff:
        ws = pa.alloc_diff_workspace(rows, heads, size, top, DEV)
        pa.pa_diff_decode(out, q.to(DEV), kc, vc, _int(table), _int(lens), lambdas=lam.to(DEV), norm=False, **kw, **ws)
    else:
        ws = pa.alloc_workspace(n, heads, size, top, DEV, num_query_tokens=rows if q_len else None)
        if kv:
            kc, vc = kc.view(torch.uint8), vc.view(torch.uint8)
        pa.pa_decode(out, q.to(DEV), kc, vc, _int(table), _int(lens), **kw, **ws)
    torch.cuda.synchronize()
    assert int(err) == 0
    got, q, lam = out.double().cpu().numpy(), q.double().numpy(), lam.double().numpy()
    absolute, relative = TOL[dtype]
    odd_outputs = 0
    for s in range(n):
        ks = k[table[s, :own[s]]].transpose(0, 2, 1, 3).reshape(-1, kh, size)
        vv = v[table[s, :own[s]]].transpose(0, 2, 1, 3).reshape(-1, kv_heads, vs)
        for r in range(start[s], start[s + 1]):
            pos = lens[s] - (start[s + 1] - r)
            lo = max(0, pos - window) if window >= 0 else 0
            if pos < 0:
                assert np.all(got[r] == 0)
                continue
            for h in range(heads):
                g = h // group

                def one(query, keys):
                    with np.errstate(invalid="ignore"):
                        z = size ** -0.5 * keys[lo:pos + 1] @ query
                        w = np.exp(z - z.max())
                        return (w / w.sum()) @ vv[lo:pos + 1, g]
                with np.errstate(invalid="ignore"):
                    want = one(q[r, h, 0], ks[:, 2 * g]) - lam[h] * one(q[r, h, 1], ks[:, 2 * g + 1]) if diff else \
                        one(q[r, h], ks[:, g])
                fine = np.isfinite(want)
                odd_outputs += int((~fine).sum())
                assert np.array_equal(np.isfinite(got[r, h]), fine), (s, r, h, np.argwhere(np.isfinite(got[r, h]) != fine)[:4])
                assert np.all(np.abs(got[r, h] - want)[fine] <= (absolute + relative * np.abs(want))[fine]), (s, r, h)
    return odd_outputs


@pytest.mark.parametrize("mode", ["v1", "v2"])
@pytest.mark.parametrize("layout", ["split", "nhd"])
@pytest.mark.parametrize("dtype,kv", TYPES)
@pytest.mark.parametrize("diff,size,group", [(False, 64, 4), (False, 128, 12), (True, 64, 3), (True, 64, 7), (True, 128, 2),
                                             (True, 128, 8)])
def test_tokens_before_the_window(diff, size, group, dtype, kv, layout, mode):
    lens = [5, 40, 700, 1037]
    for window in (0, 3, 100, 600):
        odd = [(s, t, key, value) for s, n in enumerate(lens) for t in (n - window - 2, n - window - 4, n - window - 9)
               if t >= 0 for key in (False, True) for value in (float("nan"), float("inf"))]
        assert _run(diff, dtype, kv, layout, size, 2, group, lens, None, window, odd, mode) == 0


@pytest.mark.parametrize("mode", ["v1", "v2"])
@pytest.mark.parametrize("layout", ["split", "nhd"])
@pytest.mark.parametrize("dtype,kv", TYPES)
@pytest.mark.parametrize("diff,size,group,most", [(False, 64, 2, 4), (False, 128, 4, 4), (False, 128, 1, 16), (True, 64, 1, 4),
                                                  (True, 64, 2, 4), (True, 128, 1, 8)])
def test_tokens_before_the_window_of_every_row(diff, size, group, most, dtype, kv, layout, mode):
    lens = [most, 33, 530, 1030]
    q_len = [most, most - 1, most, 2]
    for window in (1, 40, 515):
        odd = [(s, t, key, value) for s, (n, q) in enumerate(zip(lens, q_len)) for t in (n - q - window - 1, n - q - window - 6)
               if t >= 0 for key in (False, True) for value in (float("nan"), float("inf"))]
        assert _run(diff, dtype, kv, layout, size, 2, group, lens, q_len, window, odd, mode, seed=3) == 0
