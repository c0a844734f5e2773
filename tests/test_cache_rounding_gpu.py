"""GPU test of what pa_append_kv stores in an fp8 cache: the quotient with the scale,
rounded in fp32, and then to the nearest fp8 value, for every number that a 16-bit row
can hold."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import paged_kv_attention_v2_gb300 as pa  # noqa: E402
from cache_ref import cache_shapes, store_ref  # noqa: E402

DEV = "cuda:0"
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
# 0.3, 7, 0.8125, 41: the product with the reciprocal rounds 30 to 62 of the values
# to another neighbour; 1.3: every thirteenth bf16 value is a tie but for the scale's own
# rounding; powers of two; mantissas of ones; reciprocals at the ends of fp32's range
SCALES = [(0.3, 7.0), (0.8125, 41.0), (0.1, 1.9), (1.3, 1.1), (1.0, 2.0 ** -7), (3.3e-5, 1e6), (2 - 2.0 ** -23, 2.0 ** -24 - 2.0 ** -48),
          (1.5e38, 3e38), (1e-37, 2.0 ** 127)]


@pytest.mark.parametrize("layout", ["split", "nhd"])
@pytest.mark.parametrize("kv", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads", [1, 10], ids=["few", "many"])
def test_every_value_is_the_quotient(dtype, kv, layout, heads):
    size, tokens = 128, 512
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
    x = torch.where(torch.isnan(x), torch.zeros_like(x), x)  # every number and both infinities
    x = x[torch.randperm(65536, generator=torch.Generator().manual_seed(1))]
    rows = x.view(tokens, 1, size).expand(tokens, heads, size)
    slots = np.arange(tokens) + 5
    blocks = tokens // 16 + 1
    ks, vs = cache_shapes(blocks, heads, size, heads, size, layout, 1)
    key = x.to(DEV).view(tokens, 1, size).expand(tokens, heads, size)
    top = torch.finfo(FP8[kv]).max
    for scales in SCALES:
        kc, vc = torch.zeros(ks, dtype=torch.uint8, device=DEV), torch.zeros(vs, dtype=torch.uint8, device=DEV)
        pa.pa_append_kv(key, key, kc, vc, torch.from_numpy(slots.astype(np.int32)).to(DEV), layout=layout, kv_dtype=kv,
                        k_scale=scales[0], v_scale=scales[1])
        for name, c, shape, scale in (("key", kc, ks, scales[0]), ("value", vc, vs, scales[1])):
            want = (rows.float() / torch.tensor(scale, dtype=torch.float32)).clamp(-top, top).to(FP8[kv]).view(torch.uint8)
            want = store_ref(np.zeros(shape, dtype=np.uint8), want.numpy(), slots, layout, name == "key")
            got = c.cpu().numpy()
            assert np.array_equal(got, want), (name, scale, int((got != want).sum()))
