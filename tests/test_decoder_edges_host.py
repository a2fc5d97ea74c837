"""Host-side edges of the attention calls: sizes that are planned and refused
before anything is enqueued (no GPU; the pointers are never read)."""
import ctypes

import pytest

import quantized_weight_streaming_dequant_gb300 as rf

OK, INVALID, TOO_LARGE = 0, 1, 9
P = 1 << 20   # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def L():
    from quantized_weight_streaming_dequant_gb300 import build
    build.build()
    return rf.lib()


def cache(kv=1, dim=64, page=256, n_pages=10):
    return rf.KVCacheStruct(P, P, P, P, n_pages, page, kv, dim, 0)


def batch(n_tok, width, n_seq=1):
    return rf.KVBatchStruct(P, P, P, width, width, n_seq, n_tok, 0)


def workspace(L, c, b, dtype, heads, window, max_len):
    return L.rf_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(b), dtype, heads, window, max_len)


@pytest.mark.parametrize("n_tok,heads", [(1, 1), (1, 8), (500, 8)])
@pytest.mark.parametrize("dtype", [rf.F32, rf.BF16])
@pytest.mark.parametrize("window", [2 ** 31, 2 ** 62, 2 ** 63 - 600, 2 ** 63 - 1])
def test_a_window_that_hides_nothing_is_planned_like_none(L, n_tok, heads, dtype, window):
    c, b = cache(), batch(n_tok, 512)
    want = workspace(L, c, b, dtype, heads, 0, 131072)
    assert want > 0
    assert workspace(L, c, b, dtype, heads, window, 131072) == want
