"""GPU tests of what pa_diff_decode keeps when its two maps nearly cancel: the
difference is normalised, so what is lost in one map's weights or logits grows by as
much.  Against the formula in 64 bits, within the error that diff_bounds.py derives."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from diff_bounds import nearly_equal_maps, tight_ref  # noqa: E402
from diff_ref import make_case  # noqa: E402
from test_diff_gpu import TYPES, Call  # noqa: E402


def _check(c, modes):
    want, tol = tight_ref(c)
    for mode in modes:
        call = Call(c, mode).run()
        torch.cuda.synchronize()
        got = call.out.double().cpu().numpy()
        off = np.abs(got - want) / np.maximum(tol, 1e-30)
        assert int(call.err) == 0 and np.all(off <= 1), (mode, float(np.nanmax(off)), int((~(off <= 1)).sum()), off.size)


LENS = (10, 40, 513, 1500)


@pytest.mark.parametrize("layout", ["split", "nhd"])
@pytest.mark.parametrize("dtype,kv", TYPES)
@pytest.mark.parametrize("size,group", [(64, 4), (64, 8), (128, 3), (128, 5)])
def test_maps_that_nearly_cancel(dtype, kv, size, layout, group):
    for lam in (0.95, 1.0):
        _check(nearly_equal_maps(make_case(21, dtype, kv, size, layout, 2, group, LENS), lam=lam), ("v1", "v2"))


@pytest.mark.parametrize("dtype,kv", TYPES)
def test_maps_that_nearly_cancel_for_several_tokens(dtype, kv):
    _check(nearly_equal_maps(make_case(22, dtype, kv, 64, "split", 2, 2, LENS, q_len=[4, 1, 2, 3])), ("v1", "v2"))


@pytest.mark.parametrize("cap", [30.0, 64.0, 65.0, 1e4, 1e6, 1e30])
@pytest.mark.parametrize("dtype,kv", TYPES)
@pytest.mark.parametrize("group", [2, 8])
def test_softcap_of_any_size(dtype, kv, group, cap):
    """The cap's error goes by the logit: a large cap is as good as none."""
    _check(make_case(23, dtype, kv, 64, "nhd", 2, group, LENS, softcap=cap, mult=1.5), ("v1", "v2"))


@pytest.mark.parametrize("dtype,kv", TYPES)
def test_logits_beyond_the_softcap(dtype, kv):
    """Logits from far below to far above the cap."""
    for cap, mult in ((0.5, 2.0), (20.0, 4.0), (80.0, 8.0), (200.0, 8.0)):
        _check(make_case(25, dtype, kv, 64, "split", 2, 4, LENS, softcap=cap, mult=mult), ("v1", "v2"))


@pytest.mark.parametrize("dtype,kv", [("f16", None), ("bf16", "e4m3")])
def test_softcap_of_any_size_for_wide_heads_and_several_tokens(dtype, kv):
    _check(make_case(24, dtype, kv, 128, "split", 2, 2, LENS, q_len=[2, 4, 1, 3], softcap=1e6), ("v1", "v2"))
