"""GPU tests of what unusual sequences, positions and queries may do in the
cache and the attention over it."""
import numpy as np
import pytest
import torch

import quantized_weight_streaming_dequant_gb300 as rf
from decoder_helpers import Setup, by_tiles, i32, randn
from oracle import decoder as od

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_status():
    rf.device_status()
    yield
    rf.device_status()


def check_sequences(su, q, q64, dtype, which, window=0, max_len=0):
    """The rows of sequences `which` against the oracle, within its bound."""
    out = rf.attention(su.cache, su.batch, q, window=window, max_len=max_len).double().cpu().numpy()
    dim = q.shape[2]
    for s in which:
        a, b = int(su.q_start[s]), int(su.q_start[s + 1])
        ref, mag, xmag = od.attention(su.ref, su.table[s:s + 1], [su.past[s]], [0, b - a], b - a, q64[a:b], dim ** -0.5, window)
        bound = od.attention_bound(dtype, dim, su.past[s] + b - a, ref, mag, xmag)
        worst = (np.abs(out[a:b] - ref) / bound).max()
        assert worst <= 1.0, (s, worst)


# Sequences before, between and after the one that is too long; 16 heads of one
# K/V head, so that the call goes through the 128-row tiles.
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("long_at", [0, 1, 2])
def test_a_sequence_past_its_table_takes_nothing_from_the_others(dtype, window, long_at):
    rng = np.random.default_rng([21, window, long_at])
    su = Setup(rng, [192, 130, 192], [64, 64, 64], 1, 64, 64, width=4)
    assert su.table.shape[1] == 4 and by_tiles(su, 16, window)
    su.past[long_at] = 4096
    su.batch = rf.KVBatch(i32(su.table), i32(su.past), i32(su.q_start), su.n_tok)
    q, q64 = randn(rng, (su.n_tok, 16, 64), dtype, 2.0)
    check_sequences(su, q, q64, dtype, [s for s in range(3) if s != long_at], window)
    assert rf.device_status() == 1                              # the long one is reported


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("long_at", [0, 1, 2])
def test_a_sequence_longer_than_max_len_takes_nothing_from_the_others(dtype, window, long_at):
    rng = np.random.default_rng([22, window, long_at])
    past = [192, 130, 192]
    past[long_at] = 900
    su = Setup(rng, past, [64, 64, 64], 1, 64, 64)
    assert by_tiles(su, 16, window, max_len=256)
    q, q64 = randn(rng, (su.n_tok, 16, 64), dtype, 2.0)
    check_sequences(su, q, q64, dtype, [s for s in range(3) if s != long_at], window, max_len=256)


@pytest.mark.parametrize("with_q", [True, False])
def test_positions_end_at_two_to_the_31(with_q):
    """The last three positions that there are, and one that is none: it is
    skipped and reported, although the table has a page for it."""
    rng = np.random.default_rng(24)
    page, dim, width = 256, 64, 2 ** 23 + 1
    table = torch.zeros((1, width), dtype=torch.int32, device="cuda")
    table[0, -2], table[0, -1] = 1, 2
    small = od.Cache(rng.integers(-127, 128, (3, 2, page, dim)).astype(np.int8), rng.integers(-127, 128, (3, 2, page, dim)).astype(np.int8),
                     rng.integers(118, 123, (3, 2, 8)).astype(np.uint8), rng.integers(118, 123, (3, 2, 8)).astype(np.uint8))
    cache = rf.KVCache(*(torch.from_numpy(a).cuda() for a in (*small.codes, *small.scales)))
    batch = rf.KVBatch(table, i32([2 ** 31 - 3]), i32([0, 4]), 4)
    k, v = randn(rng, (4, 2, dim))[0], randn(rng, (4, 2, dim))[0]
    q, q64 = randn(rng, (4, 4, dim))
    out = torch.full_like(q, 7.0)
    rf.kv_append(cache, batch, k, v, **(dict(q=q, q_out=out) if with_q else {}))
    assert rf.device_status() == 1 and rf.device_status() == rf.OK
    if with_q:
        assert torch.equal(out[:3], q[:3]) and (out[3] == 7.0).all()
    small.append(np.array([[1]]), [page - 3], [0, 3], k.cpu().numpy(), v.cpu().numpy())
    for got, want in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), small.codes + small.scales):
        assert np.array_equal(got.cpu().numpy(), want)
    kr, vr = rf.kv_read(cache, batch)
    assert rf.device_status() == 1
    for t in range(3):
        assert np.array_equal(kr[t].double().cpu().numpy(), small.values([1], page - 3 + t, 0))
        assert np.array_equal(vr[t].double().cpu().numpy(), small.values([1], page - 3 + t, 1))
    assert not kr[3].any() and not vr[3].any()
    got = rf.attention(cache, batch, q, window=8).double().cpu().numpy()
    assert rf.device_status() == 1
    ref, mag, xmag = od.attention(small, np.array([[1]]), [page - 3], [0, 3], 3, q64[:3], dim ** -0.5, 8)
    assert (np.abs(got[:3] - ref) <= od.attention_bound("float32", dim, 8, ref, mag, xmag)).all()


@pytest.mark.parametrize("past,new,heads", [(6000, 1, 4), (4000, 40, 4), (300, 60, 32)])
def test_attention_on_a_busy_stream_keeps_its_workspace(past, new, heads):
    """The current stream allocates and fills blocks of the workspace's size
    while the calls still wait on a stream of their own."""
    rng = np.random.default_rng([25, past])
    su = Setup(rng, [past], [new], 1, 64, 64)
    q, _ = randn(rng, (new, heads, 64))
    want = rf.attention(su.cache, su.batch, q)
    size = rf.attention_workspace(su.cache, su.batch, q)
    size = 0 if size is None else size.numel()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = [rf.attention(su.cache, su.batch, q, stream=handle) for _ in range(3)]
        fill = [torch.full((max(size, 1),), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        fill += [torch.full_like(q, 7.0) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(g, want) for g in got)
        assert all((f == f.flatten()[0]).all() for f in fill)


# One token and a chunk in one part (rows), rows in several parts, tiles in one
# part and in several.
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("past,new,heads", [(0, 1, 4), (150, 3, 4), (6000, 1, 4), (300, 60, 32), (4000, 40, 4)])
def test_an_infinite_query_gives_nan_whatever_the_signs_of_its_scores(dtype, past, new, heads):
    """Scores that are all minus infinity are seen all the same: such a row is
    not one that sees nothing."""
    rng = np.random.default_rng([23, past, new])
    su = Setup(rng, [past], [new], 1, 64, 64)
    su.ref.codes[0][..., 7] = -np.abs(su.ref.codes[0][..., 7]) - (su.ref.codes[0][..., 7] == 0)
    su.upload()
    q, q64 = randn(rng, (new, heads, 64), dtype)
    clean = rf.attention(su.cache, su.batch, q)
    q[0, 1, 7] = float("inf")
    q[new - 1, 2, 7] = float("-inf")
    out = rf.attention(su.cache, su.batch, q)
    hit = torch.zeros((new, heads), dtype=torch.bool, device="cuda")
    hit[0, 1] = hit[new - 1, 2] = True
    assert torch.isnan(out[hit]).all()
    assert torch.equal(out[~hit], clean[~hit])
