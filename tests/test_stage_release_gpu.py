"""A page's shared-memory stage goes back to the producer only after the page's
last read has returned.

Batches in which some CTAs zero the unused slots of partial pages (a burst of
conflicting shared-memory stores) while their neighbours on the same SM stream
whole partitions: a stage handed back too early is refilled under reads that are
still queued, which showed as different outputs from one call to the next (57 of
5000 calls, fp32 caches in the split layout).  The kernels are deterministic, so
every call must give the same bits.
"""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import paged_kv_attention_v2_gb300 as pa  # noqa: E402

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.mark.parametrize("dtype,kv,layout,group,calls", [
    ("f32", None, "split", 8, 3000), ("f32", None, "nhd", 8, 500), ("f32", None, "split", 16, 500),
    ("f16", None, "split", 8, 500), ("bf16", None, "nhd", 16, 500), ("f16", "e4m3", "split", 8, 500),
    ("bf16", "e5m2", "nhd", 16, 500)])
def test_calls_repeat_bit_for_bit(dtype, kv, layout, group, calls):
    n, kvh, d, longest, dev = 40, 4, 128, 17000, "cuda:0"
    lens = np.full(n, 97)  # one token in the last page: fifteen slots zeroed
    lens[0], lens[-1] = longest, longest - 777
    rng, gen = np.random.default_rng(1), torch.Generator(device=dev).manual_seed(5)
    own = -(-lens // 16)
    ids = rng.permutation(int(own.sum()))
    table = np.zeros((n, -(-longest // 16)), dtype=np.int32)
    for s, end in enumerate(np.cumsum(own)):
        table[s, :own[s]] = ids[end - own[s]:end]
    ct = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}.get(kv, TORCH[dtype])
    x = 16 // ct.itemsize
    ks, vs = ((len(ids), kvh, d // x, 16, x), (len(ids), kvh, d, 16)) if layout == "split" else ((len(ids), kvh, 16, d),) * 2
    k, v = (torch.randn(s, generator=gen, device=dev).to(ct) for s in (ks, vs))
    if kv:
        k, v = k.view(torch.uint8), v.view(torch.uint8)
    q = torch.randn((n, kvh * group, d), generator=gen, device=dev).to(TORCH[dtype])
    tensors = (k, v, torch.from_numpy(table).to(dev), torch.from_numpy(lens.astype(np.int32)).to(dev))
    ws = pa.alloc_workspace(n, kvh * group, d, longest, dev)
    out, first, differ = torch.empty_like(q), None, torch.zeros((), device=dev)
    for _ in range(calls):
        pa.pa_decode(out, q, *tensors, num_kv_heads=kvh, scale=d ** -0.5, max_seq_len=longest, mode="v2", layout=layout,
                     kv_dtype=kv, **ws)
        if first is None:
            first = out.clone()
        else:
            differ += (out != first).any()
    assert int(differ) == 0, f"{int(differ)} of {calls} calls differ from the first"
