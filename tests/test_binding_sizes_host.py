"""Host-side checks (no GPU) of pa_decode's Python binding: sizes that do not fit the argument struct are
refused with the library's status, and not taken modulo 2^32; a window of any size is taken."""
import pytest

import paged_kv_attention_v2_gb300 as pa
from paged_kv_attention_v2_gb300 import _abi, evict

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def lib():
    from paged_kv_attention_v2_gb300 import build
    build.build()


def _args(**over):
    h = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    kw = {**dict(num_kv_heads=2, scale=0.1, max_seq_len=40), **over}
    return pa.make_args(h(3, 4, 64), h(3, 4, 64), h(7, 2, 8, 16, 8), h(7, 2, 64, 16), i(3, 3), i(3), **kw)


@pytest.mark.parametrize("over", [dict(max_seq_len=2 ** 31), dict(max_seq_len=2 ** 32 + 40), dict(max_seq_len=-2 ** 31 - 1)])
def test_sizes_beyond_32_bits(over):
    with pytest.raises(pa.PaDecodeError) as e:
        _args(**over)
    assert e.value.status == _abi.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("over", [dict(max_seq_len=40.0), dict(max_seq_len="40"), dict(scale="0.1")])
def test_what_is_no_number(over):
    with pytest.raises(TypeError):
        _args(**over)


@pytest.mark.parametrize("window,sliding", [(-1, 0), (0, 1), (99, 100), (2 ** 31 - 2, 2 ** 31 - 1), (2 ** 31 - 1, 0), (2 ** 40, 0)])
def test_windows_over_any_length_are_none(window, sliding):
    assert _args(window_left=window).sliding_window == sliding
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    a = evict.make_weights_args(torch.zeros(7, 2, 16), torch.zeros(3, 4, 64).half(), torch.zeros(7, 2, 16, 64).half(), i(3, 3), i(3),
                                torch.zeros(3, 4, 1), torch.zeros(3, 4, 1), num_kv_heads=2, scale=0.1, max_seq_len=40, layout="nhd",
                                window_left=window, relative_max=True)
    assert a.sliding_window == sliding and a.relative_max == 1


def test_what_fits_is_packed():
    a = _args(max_seq_len=2 ** 31 - 1, window_left=2 ** 31 - 2, relative_max=True, scale=1e39)
    assert (a.max_seq_len, a.sliding_window, a.relative_max, a.scale) == (2 ** 31 - 1, 2 ** 31 - 1, 1, float("inf"))
    assert _args().relative_max == 0
