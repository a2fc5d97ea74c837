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


def test_the_plan_of_a_call_is_checked_and_laid_out_on_the_host(L):
    p = rf.AttentionPlan()
    ask = lambda c, b, heads=8, window=0, max_len=0, dtype=rf.F32, out=p: L.rf_debug_attention_plan(  # noqa: E731
        ctypes.byref(c), ctypes.byref(b), dtype, heads, window, max_len, ctypes.byref(out) if out is not None else None)
    assert ask(cache(), batch(1, 4), out=None) == INVALID
    assert ask(cache(dim=72), batch(1, 4)) == INVALID and ask(cache(), batch(1, 4), window=-1) == INVALID
    assert ask(cache(), batch(1, 4), heads=4097) == TOO_LARGE and ask(cache(), batch(1, 4), dtype=5) == 2
    assert ask(cache(), batch(0, 4)) == OK and (p.tiles, p.parts, p.reserved) == (0, 0, 0)
    assert ask(cache(), batch(1, 2)) == OK
    assert (p.tiles, p.parts, p.part_positions, p.item_tokens, p.head_tiles) == (0, 1, 512, 1, 1)
    assert ask(cache(), batch(1, 64)) == OK and p.tiles == 0 and p.parts > 1 and p.parts * p.part_positions >= 64 * 256
    assert ask(cache(), batch(2000, 8, 2)) == OK
    assert p.tiles == 1 and p.item_tokens == 32 and p.head_tiles == 1 and p.parts * p.part_positions >= 2048
    assert ask(cache(dim=256), batch(2000, 8, 2)) == OK and p.item_tokens == 16


@pytest.mark.parametrize("heads,kv", [(1, 1), (8, 1), (8, 2), (64, 8), (130, 1)])
@pytest.mark.parametrize("window", [0, 33, 1000])
def test_the_tests_rule_of_the_path_is_the_librarys(L, heads, kv, window):
    """The GPU tests say with `by_tiles` which path a case takes."""
    import types

    from decoder_helpers import by_tiles
    p = rf.AttentionPlan()
    took = set()
    for n_tok in (1, 2, 3, 11, 12, 13, 24, 95, 96, 97, 192, 500, 4000):
        for n_seq in (1, 2, 7):
            for width in (1, 9, 40, 500):
                for max_len in (0, 300, 2500):
                    c, b = cache(kv), batch(n_tok, width, n_seq)
                    su = types.SimpleNamespace(n_tok=n_tok, past=[0] * n_seq, table=types.SimpleNamespace(shape=(n_seq, width)),
                                               ref=types.SimpleNamespace(heads=kv, page=256))
                    assert L.rf_debug_attention_plan(ctypes.byref(c), ctypes.byref(b), rf.F32, heads, window, max_len, ctypes.byref(p)) == OK
                    capped = min(max_len, 256 * width)          # the tests pass no max_len past the table
                    assert bool(p.tiles) == by_tiles(su, heads, window, capped), (n_tok, n_seq, width, max_len)
                    took.add(p.tiles)
    assert took == {0, 1}


def test_the_most_tokens_of_a_call_are_counted_in_64_bits(L):
    p = rf.AttentionPlan()
    c, b = cache(), batch(2 ** 31 - 1, 4, 65536)
    assert L.rf_debug_attention_plan(ctypes.byref(c), ctypes.byref(b), rf.F32, 1, 0, 0, ctypes.byref(p)) == OK
    assert p.tiles == 1                                         # 32,768 tokens a sequence
