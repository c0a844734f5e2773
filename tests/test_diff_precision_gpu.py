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
