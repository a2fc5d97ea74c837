"""GPU tests of the operators between the projections: fused norms, the paged
8-bit KV cache and attention over it, each against the fp64 oracle."""
import numpy as np
import pytest
import torch

import quantized_weight_streaming_dequant_gb300 as rf
from decoder_helpers import DTYPES, TORCH, Setup, by_tiles, check_attention, i32, randn, strided
from oracle import decoder as od

pytestmark = pytest.mark.gpu

HALF_ULP = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


@pytest.fixture(autouse=True)
def clean_status():
    rf.device_status()
    yield
    rf.device_status()


# ------------------------------------------------------------------- norms
def norm_check(dtype, x, x64, res, res64, post, gate, scale, weight, eps=1e-5, **kw):
    """r within a few fp32 roundings of its terms; y within the sums of squares'
    (up to 32 sequential terms and a tree: 64 * 2^-24) and r's."""
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    r, y = rf.norm_residual(res, x, post_weight=dev(post), gate=dev(gate), scale=scale, weight=dev(weight), eps=eps, **kw)
    scale = np.float32(scale)
    r64, y64 = od.norm_residual(x64, res64, post, gate, scale, weight, np.float32(eps))
    parts = np.abs(r64 - (0 if res64 is None else res64)) + (0 if res64 is None else np.abs(res64))
    tol = 2.0 ** -17 * parts
    inv = 1 / np.sqrt(np.mean(r64 * r64, -1, keepdims=True) + eps)
    tol_y = (tol + 2.0 ** -17 * np.abs(r64)) * inv * (1 if weight is None else np.abs(weight))
    # the whole row's sum of squares moves with the whole row's error
    tol_y = tol_y + 2.0 ** -17 * np.abs(y64)
    for got, want, t in ((r, r64, tol), (y, y64, tol_y)):
        if got is not None:
            g = got.double().cpu().numpy()
            ok = np.abs(g - want) <= t + HALF_ULP[dtype] * np.abs(want) * 1.01 + (0 if dtype != "float16" else 2.0 ** -25)
            assert ok.all(), (np.argwhere(~ok)[:4], g[~ok][:4], want[~ok][:4])
    return r, y


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n_tok,n", [(1, 1), (3, 7), (2, 64), (1, 4096), (5, 2880), (300, 129), (400, 1024), (2, 16392),
                                     (1, 32768), (3, 32767)])
def test_norm_residual(dtype, n_tok, n):
    rng = np.random.default_rng([n_tok, n])
    x, x64 = randn(rng, (n_tok, n), dtype)
    res, res64 = randn(rng, (n_tok, n), dtype, 3.0)
    f = lambda: (1 + 0.3 * rng.standard_normal(n)).astype(np.float32)  # noqa: E731
    norm_check(dtype, x, x64, res, res64, f(), f(), 0.7, f())
    norm_check(dtype, x, x64, res, res64, None, None, -1.0, None)


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_parts_that_drop_out(dtype):
    rng = np.random.default_rng(5)
    x, x64 = randn(rng, (4, 96), dtype)
    res, res64 = randn(rng, (4, 96), dtype)
    w = (1 + 0.1 * rng.standard_normal(96)).astype(np.float32)
    norm_check(dtype, None, None, res, res64, w, w, 3.0, w)
    norm_check(dtype, x, x64, None, None, w, None, 0.5, w)
    gate = rng.standard_normal((4, 96)).astype(np.float32)
    norm_check(dtype, x, x64, res, res64, None, gate, 1.0, w)
    r, y = norm_check(dtype, x, x64, res, res64, w, None, 1.0, None, norm=False)
    assert y is None
    zero = torch.zeros((2, 96), dtype=TORCH[dtype], device="cuda")
    r, y = rf.norm_residual(zero, zero)
    assert not r.any() and not y.any()
    empty = zero[:0]
    r, y = rf.norm_residual(empty, empty)
    assert r.shape == (0, 96) and y.shape == (0, 96)


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_strides_and_in_place(dtype):
    rng = np.random.default_rng(6)
    x, x64 = randn(rng, (6, 256), dtype)
    res, res64 = randn(rng, (6, 256), dtype)
    w = (1 + 0.1 * rng.standard_normal(256)).astype(np.float32)
    want = norm_check(dtype, x, x64, res, res64, w, w, 1.5, w)
    for off, width in ((0, 320), (3, 263), (8, 264)):          # aligned, odd, aligned with a shift
        bx = torch.full((6, width), float("nan"), dtype=TORCH[dtype], device="cuda")
        br = bx.clone()
        vx, vr = bx[:, off:off + 256], br[:, off:off + 256]
        vx.copy_(x), vr.copy_(res)
        got = norm_check(dtype, vx, x64, vr, res64, w, w, 1.5, w, residual_out=vr, y=vx)
        assert got[0].data_ptr() == vr.data_ptr()
        # the wide and the narrow accesses order the sums differently: equal within the bound (checked above)
        assert torch.allclose(got[1].float(), want[1].float(), rtol=2e-2 if dtype != "float32" else 1e-5, atol=1e-5)
        assert torch.isnan(bx[:, off + 256:]).all() and torch.isnan(br[:, :off]).all()


def test_norm_nan_and_inf_stay_in_their_row():
    x = torch.ones((3, 64), device="cuda")
    x[1, 5] = float("nan")
    r, y = rf.norm_residual(None, x)
    assert torch.isfinite(y[0]).all() and torch.isnan(y[1]).all() and torch.isfinite(y[2]).all()
    x[1, 5] = float("inf")
    r, y = rf.norm_residual(None, x)
    assert torch.isnan(y[1, 5]) and not y[1, :5].any() and torch.isfinite(y[2]).all()


# ------------------------------------------------------------------ append
def tables(n_pos, rot):
    if rot == 0:
        return None, None
    a = np.arange(n_pos)[:, None] * (10000.0 ** (-np.arange(rot // 2) / (rot // 2)))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def append_check(su, dtype, rng, rot, style, heads, n_pos=None, stretch=0, scale=1.0):
    kv, dim = su.ref.heads, su.ref.dim
    k, k64 = randn(rng, (su.n_tok, kv, dim), dtype, scale)
    v, v64 = randn(rng, (su.n_tok, kv, dim), dtype, scale)
    q, q64 = randn(rng, (su.n_tok, heads, dim), dtype)
    top = max(p + n for p, n in zip(su.past, su.new))
    cos, sin = tables(n_pos or top, rot)
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    if stretch:
        k, v, q = strided(k, stretch, stretch), strided(v, 1, 0), strided(q, 0, stretch)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    got = rf.kv_append(su.cache, su.batch, k, v, q=q, q_out=out, cos=dev(cos), sin=dev(sin), rope=style)
    pairs = style == rf.ROPE_PAIRS
    kr, qr = np.array(k64, np.float32), np.full(q64.shape, 7.0, np.float32)
    for s in range(len(su.past)):
        for t in range(su.q_start[s], su.q_start[s + 1]):
            p = su.past[s] + t - su.q_start[s]
            c, d = (None, None) if rot == 0 else (cos[p], sin[p])
            kr[t], qr[t] = od.rotate(k64[t], c, d, pairs), od.rotate(q64[t], c, d, pairs)
    assert torch.equal(got.cpu(), torch.from_numpy(qr).to(TORCH[dtype]))
    su.ref.append(su.table, su.past, su.q_start, kr, np.array(v64, np.float32))
    su.same_cache()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim,rot,style,page,heads,kv", [
    (64, 64, rf.ROPE_HALF, 64, 8, 2), (128, 128, rf.ROPE_PAIRS, 32, 4, 4), (128, 64, rf.ROPE_HALF, 128, 5, 1),
    (80, 32, rf.ROPE_PAIRS, 256, 6, 3), (16, 8, rf.ROPE_HALF, 32, 1, 1), (256, 256, rf.ROPE_HALF, 64, 2, 1),
    (112, 0, rf.ROPE_HALF, 64, 7, 7)])
def test_append_codes_are_exact(dtype, dim, rot, style, page, heads, kv):
    rng = np.random.default_rng([dim, rot])
    su = Setup(rng, [0, 37, 95, 31, 64], [70, 1, 2, 33, 0], kv, dim, page)
    append_check(su, dtype, rng, rot, style, heads)
    assert rf.device_status() == rf.OK


@pytest.mark.parametrize("new", [[1] * 9, [200], [3, 0, 150, 1]])
def test_append_token_by_token_and_in_chunks(new):
    rng = np.random.default_rng(len(new))
    past = [int(p) for p in rng.integers(0, 130, len(new))]
    su = Setup(rng, past, new, 2, 64, 64, width=6)
    append_check(su, "float32", rng, 64, rf.ROPE_HALF, 4, stretch=3)
    # further tokens onto the same blocks, growing: units double, held codes are re-rounded
    for step in range(3):
        su.past = [p + n for p, n in zip(su.past, su.new)]
        su.new = [1] * len(new)
        su.q_start = np.arange(len(new) + 1, dtype=np.int32)
        su.n_tok = len(new)
        su.batch = rf.KVBatch(i32(su.table), i32(su.past), i32(su.q_start), su.n_tok)
        append_check(su, "float32", rng, 64, rf.ROPE_HALF, 4, stretch=4, scale=2.0 ** (2 * step))


def test_append_special_values():
    rng = np.random.default_rng(9)
    su = Setup(rng, [3, 40], [2, 2], 1, 32, 32)
    k, _ = randn(rng, (4, 1, 32))
    v, _ = randn(rng, (4, 1, 32))
    k[0, 0, 3], v[2, 0, 7], k[3, 0, 0] = float("nan"), float("-inf"), 2.0 ** 60
    v[0] = 0
    rf.kv_append(su.cache, su.batch, k, v)
    su.ref.append(su.table, su.past, su.q_start, k.cpu().numpy(), v.cpu().numpy())
    su.same_cache()
    kr, vr = rf.kv_read(su.cache, su.batch)
    assert torch.isnan(kr).all() and torch.isfinite(vr[:2]).all() and torch.isnan(vr[2:]).all()
    # a block's first token starts it afresh
    su.past, su.new, su.q_start, su.n_tok = [0, 32], [1, 1], np.array([0, 1, 2], np.int32), 2
    su.batch = rf.KVBatch(i32(su.table), i32(su.past), i32(su.q_start), 2)
    k, v = torch.zeros((2, 1, 32), device="cuda"), torch.ones((2, 1, 32), device="cuda")
    rf.kv_append(su.cache, su.batch, k, v)
    su.ref.append(su.table, su.past, su.q_start, k.cpu().numpy(), v.cpu().numpy())
    su.same_cache()


def test_tokens_without_a_page_are_skipped_and_reported():
    rng = np.random.default_rng(10)
    su = Setup(rng, [0, 64, 5], [1, 1, 1], 2, 64, 64, pad_tokens=3)
    su.table[0, 0], su.table[1, 1] = 10 ** 6, -5
    su.batch = rf.KVBatch(i32(su.table), i32(su.past), i32(su.q_start), su.n_tok)
    append_check(su, "float32", rng, 64, rf.ROPE_HALF, 4)
    assert rf.device_status() == 1 and rf.device_status() == rf.OK
    kr, vr = rf.kv_read(su.cache, su.batch)
    assert not kr[:2].any() and not kr[3:].any() and kr[2].any()
    assert rf.device_status() == 1
    q, q64 = randn(rng, (su.n_tok, 4, 64))
    out = check_attention(su, q, q64, "float32")
    assert not out[0].any() and out[1].any() and not out[3:].any()
    assert rf.device_status() == 1
    # a negative past and a position past the table
    su.past = [-3, 4096, 5]
    su.batch = rf.KVBatch(i32(su.table), i32(su.past), i32(su.q_start), su.n_tok)
    rf.kv_append(su.cache, su.batch, *(randn(rng, (su.n_tok, 2, 64))[0] for _ in range(2)))
    out = rf.attention(su.cache, su.batch, q)
    assert not out[0].any() and rf.device_status() == 1


def test_rotation_past_its_tables_is_skipped_and_reported():
    rng = np.random.default_rng(11)
    su = Setup(rng, [0], [70], 1, 64, 64)
    k, v = randn(rng, (70, 1, 64))[0], randn(rng, (70, 1, 64))[0]
    cos, sin = tables(40, 64)
    rf.kv_append(su.cache, su.batch, k, v, cos=torch.from_numpy(cos).cuda(), sin=torch.from_numpy(sin).cuda())
    assert rf.device_status() == 1
    kr = np.stack([od.rotate(k[t].cpu().numpy(), cos[t], sin[t], False) for t in range(40)])
    su.ref.append(su.table, [0], [0, 40], kr, v[:40].cpu().numpy())
    su.same_cache()


@pytest.mark.parametrize("dim,page", [(64, 32), (80, 256), (256, 64)])
def test_read_gives_the_held_values(dim, page):
    rng = np.random.default_rng(dim)
    su = Setup(rng, [0, 33, 7], [40, 0, 5], 3, dim, page, pad_tokens=1)
    kr, vr = rf.kv_read(su.cache, su.batch)
    for s in range(3):
        for t in range(su.q_start[s], su.q_start[s + 1]):
            p = su.past[s] + t - su.q_start[s]
            assert np.array_equal(kr[t].double().cpu().numpy(), su.ref.values(su.table[s], p, 0))
            assert np.array_equal(vr[t].double().cpu().numpy(), su.ref.values(su.table[s], p, 1))
    assert not kr[-1].any() and not vr[-1].any()


# --------------------------------------------------------------- attention
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim,heads,kv,page", [
    (64, 8, 1, 32), (64, 6, 2, 64), (128, 4, 4, 128), (128, 16, 2, 32), (128, 20, 1, 64), (80, 5, 5, 256), (16, 2, 1, 32),
    (48, 3, 1, 32), (112, 14, 2, 64), (144, 9, 1, 32), (256, 8, 2, 64), (240, 2, 2, 32)])
def test_attention_single_tokens(dtype, dim, heads, kv, page):
    rng = np.random.default_rng([dim, heads])
    past = [0, 1, 31, 32, 33, 260, 700]
    su = Setup(rng, past, [1] * len(past), kv, dim, page)
    q, q64 = randn(rng, (su.n_tok, heads, dim), dtype, 2.0)
    check_attention(su, q, q64, dtype)
    sinks = rng.standard_normal(heads).astype(np.float32)
    check_attention(su, q, q64, dtype, scale=0.2, window=40, sinks=sinks, max_len=701)
    assert rf.device_status() == rf.OK


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [[2, 5, 1, 0, 9], [70, 3], [1, 1, 40]])
@pytest.mark.parametrize("dim,heads,kv", [(64, 8, 1), (128, 4, 2), (128, 9, 3), (256, 4, 2)])
def test_attention_short_chunks(dtype, new, dim, heads, kv):
    rng = np.random.default_rng([dim, len(new)])
    su = Setup(rng, [int(p) for p in rng.integers(0, 200, len(new))], new, kv, dim, 64, pad_tokens=2)
    q, q64 = randn(rng, (su.n_tok, heads, dim), dtype, 2.0)
    out = check_attention(su, q, q64, dtype)
    assert not out[-2:].any()
    check_attention(su, q, q64, dtype, window=33)
    check_attention(su, q, q64, dtype, window=1)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_long_rows_are_split_and_joined(dtype):
    rng = np.random.default_rng(12)
    su = Setup(rng, [20000], [1], 1, 64, 64)
    q, q64 = randn(rng, (1, 8, 64), dtype, 2.0)
    a = check_attention(su, q, q64, dtype, sinks=rng.standard_normal(8).astype(np.float32))
    b = check_attention(su, q, q64, dtype, sinks=None, max_len=20001)
    assert rf.attention_workspace(su.cache, su.batch, q, 20001) is not None
    assert not torch.equal(a, b)
    c = rf.attention(su.cache, su.batch, q, max_len=20001)
    assert torch.equal(b, c)                                    # the order of the joins is fixed


def test_attention_nan_blocks_reach_only_rows_that_see_them():
    rng = np.random.default_rng(13)
    su = Setup(rng, [200, 90], [1, 1], 2, 64, 32)
    su.ref.scales[0][su.table[0, 2], 1] = 255                   # keys 64..95 of sequence 0, head 1
    su.ref.scales[1][su.table[1, 0], 0] = 255                   # values 0..31 of sequence 1, head 0
    su.upload()
    q, q64 = randn(rng, (2, 4, 64))
    out = check_attention(su, q, q64, "float32")
    assert torch.isnan(out[0, 2:]).all() and torch.isfinite(out[0, :2]).all()
    out = check_attention(su, q, q64, "float32", window=59)     # positions 142.. and 32..: outside
    assert torch.isfinite(out).all()


def test_attention_extreme_scores_and_units():
    rng = np.random.default_rng(14)
    su = Setup(rng, [150], [1], 1, 64, 32, scales=(88, 160))    # units from 2^-39 to 2^32
    q, q64 = randn(rng, (1, 2, 64), "float32", 2.0 ** -36)
    check_attention(su, q, q64, "float32")
    su = Setup(rng, [150], [1], 1, 64, 32)
    q, q64 = randn(rng, (1, 2, 64), "float32", 200.0)           # one position takes nearly all
    check_attention(su, q, q64, "float32")
    check_attention(su, q, q64, "float32", scale=0.0)           # all alike
    check_attention(su, q, q64, "float32", scale=-0.1)
    check_attention(su, 0 * q, 0 * q64, "float32", sinks=np.array([200.0, -200.0], np.float32))
    q[0, 1, 5] = float("nan")
    out = rf.attention(su.cache, su.batch, q)
    assert torch.isnan(out[0, 1]).all() and torch.isfinite(out[0, 0]).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_strides_streams_and_chains(dtype):
    rng = np.random.default_rng(15)
    su = Setup(rng, [64, 300, 7], [1, 1, 30], 2, 128, 64)
    q, q64 = randn(rng, (su.n_tok, 8, 128), dtype)
    want = check_attention(su, q, q64, dtype)
    for pad in ((2, 0), (0, 8), (1, 3)):
        qs, out = strided(q, *pad), strided(torch.zeros_like(q), *pad)
        rf.attention(su.cache, su.batch, qs, out=out)
        assert torch.equal(out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rf.attention(su.cache, su.batch, q, stream=side)
    with torch.cuda.stream(side):
        got2 = rf.attention(su.cache, su.batch, q, flags=rf.CHAIN)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(got2, want)


def test_a_captured_step_replays_with_other_lengths():
    """Lengths and pages are read by the kernels: one capture serves a decode loop."""
    rng = np.random.default_rng(16)
    su = Setup(rng, [30, 61], [1, 1], 2, 64, 64, width=3, spare=8)
    for s in range(2):                                          # give every entry a page
        for i in range(3):
            if su.table[s, i] < 0:
                free = set(range(su.ref.n_pages)) - set(su.table[su.table >= 0].tolist())
                su.table[s, i] = min(free)
    past = i32(su.past)
    batch = rf.KVBatch(i32(su.table), past, i32(su.q_start), 2)
    cos, sin = tables(192, 64)
    dc, ds = torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda()
    k, v = (torch.zeros((2, 2, 64), device="cuda") for _ in range(2))
    q, qr, out = (torch.zeros((2, 4, 64), device="cuda") for _ in range(3))
    ws = rf.attention_workspace(su.cache, batch, q)

    def step():
        rf.kv_append(su.cache, batch, k, v, q=q, q_out=qr, cos=dc, sin=ds)
        rf.attention(su.cache, batch, qr, out=out, workspace=ws, flags=rf.CHAIN)
        past.add_(1)

    keep = [t.clone() for t in (su.cache.k, su.cache.v, su.cache.k_scale, su.cache.v_scale)]
    step()                                                      # first use outside a capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, o in zip((su.cache.k, su.cache.v, su.cache.k_scale, su.cache.v_scale), keep):
        t.copy_(o)
    past.copy_(i32(su.past))
    for i in range(5):
        for t in (k, v, q):
            t.copy_(randn(rng, t.shape)[0])
        graph.replay()
        torch.cuda.synchronize()
        now = [p + i for p in su.past]
        kr = np.stack([od.rotate(k[s].cpu().numpy(), cos[now[s]], sin[now[s]], False) for s in range(2)])
        qrot = np.stack([od.rotate(q[s].cpu().numpy(), cos[now[s]], sin[now[s]], False) for s in range(2)])
        su.ref.append(su.table, now, su.q_start, kr, v.cpu().numpy())
        ref, mag, xmag = od.attention(su.ref, su.table, now, su.q_start, 2, qrot, 64 ** -0.5)
        assert (np.abs(out.double().cpu().numpy() - ref) <= od.attention_bound("float32", 64, 200, ref, mag, xmag)).all()
    su.same_cache()
    assert rf.device_status() == rf.OK


def test_many_pages_pass_32_bit_offsets():
    """A page whose codes lie beyond 2^32 bytes."""
    n_pages, dim, page = 2 ** 20 + 40, 64, 64
    cache = rf.KVCache.empty(n_pages, 1, page, dim)             # 4.3 GB of keys
    table = i32([[n_pages - 1, 3, n_pages - 7]])
    rng = np.random.default_rng(17)
    k, v = randn(rng, (150, 1, dim))[0], randn(rng, (150, 1, dim))[0]
    q, q64 = randn(rng, (150, 2, dim))
    batch = rf.KVBatch(table, i32([0]), i32([0, 150]), 150)
    rf.kv_append(cache, batch, k, v)
    small = od.Cache(np.zeros((3, 1, page, dim), np.int8), np.zeros((3, 1, page, dim), np.int8),
                     np.zeros((3, 1, 2), np.uint8), np.zeros((3, 1, 2), np.uint8))
    small.append(np.array([[0, 1, 2]]), [0], [0, 150], k.cpu().numpy(), v.cpu().numpy())
    kr, vr = rf.kv_read(cache, batch)
    for t in (0, 63, 64, 128, 149):
        assert np.array_equal(kr[t].double().cpu().numpy(), small.values([0, 1, 2], t, 0))
    out = rf.attention(cache, batch, q)
    ref, mag, xmag = od.attention(small, np.array([[0, 1, 2]]), [0], [0, 150], 150, q64, 0.125)
    assert (np.abs(out.double().cpu().numpy() - ref) <= od.attention_bound("float32", 64, 150, ref, mag, xmag)).all()
    assert rf.device_status() == rf.OK


# ------------------------------------------------------------- long chunks
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim,heads,kv,page,past,new", [
    (128, 4, 1, 64, [0], [400]), (64, 8, 1, 32, [0, 77, 3], [129, 200, 64]), (128, 2, 2, 128, [900], [600]),
    (80, 5, 1, 256, [130, 0], [190, 331]), (16, 3, 1, 32, [0], [430]), (112, 7, 1, 64, [440], [175]),
    (64, 130, 1, 64, [1400], [3]), (128, 20, 1, 32, [0, 900], [40, 7]), (64, 64, 2, 64, [0, 10, 700, 0], [0, 5, 2, 60]),
    (256, 4, 1, 64, [0, 30], [290, 270]), (144, 6, 2, 32, [100], [430]), (240, 5, 1, 128, [900, 0], [40, 150])])
def test_attention_long_chunks(dtype, dim, heads, kv, page, past, new):
    rng = np.random.default_rng([dim, heads, sum(new)])
    su = Setup(rng, past, new, kv, dim, page, pad_tokens=3)
    assert by_tiles(su, heads)
    q, q64 = randn(rng, (su.n_tok, heads, dim), dtype, 2.0)
    out = check_attention(su, q, q64, dtype)
    assert not out[-3:].any()
    sinks = rng.standard_normal(heads).astype(np.float32)
    check_attention(su, q, q64, dtype, scale=-0.15, window=37, sinks=sinks, max_len=max(p + n for p, n in zip(past, new)))
    assert rf.device_status() == rf.OK


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention_long_chunks_split_and_joined(dtype, dim):
    rng = np.random.default_rng(dim)
    su = Setup(rng, [4000], [40], 1, dim, 64, pad_tokens=1)
    assert by_tiles(su, 4, max_len=4040) and not by_tiles(su, 4, window=1000)
    q, q64 = randn(rng, (su.n_tok, 4, dim), dtype, 2.0)
    a = check_attention(su, q, q64, dtype, max_len=4040)
    assert torch.equal(a, rf.attention(su.cache, su.batch, q, max_len=4040))
    check_attention(su, q, q64, dtype, window=1000, sinks=np.array([0.5, -1.0, 2.0, 0.0], np.float32))
    check_attention(su, q, q64, dtype, scale=0.0)


def test_attention_long_chunks_hide_missing_pages_and_nan_blocks():
    rng = np.random.default_rng(18)
    su = Setup(rng, [600], [500], 2, 64, 32)
    assert by_tiles(su, 4) and by_tiles(su, 4, window=150)
    su.table[0, 3] = -1                                         # positions 96..127 have no page
    su.ref.scales[1][su.table[0, 0], 1] = 255                   # values 0..31, head 1
    su.upload()
    q, q64 = randn(rng, (su.n_tok, 4, 64))
    out = check_attention(su, q, q64, "float32")
    assert torch.isnan(out[:, 2:]).all() and torch.isfinite(out[:, :2]).all()
    assert rf.device_status() == 1
    out = check_attention(su, q, q64, "float32", window=150)    # the first row sees positions 451..
    assert torch.isfinite(out).all()


def test_attention_long_chunks_strides_streams_and_chains():
    rng = np.random.default_rng(19)
    su = Setup(rng, [64, 600], [290, 270], 2, 128, 64)
    assert by_tiles(su, 8)
    for dtype in DTYPES:
        q, q64 = randn(rng, (su.n_tok, 8, 128), dtype)
        want = check_attention(su, q, q64, dtype)
        for pad in ((2, 0), (0, 8), (1, 3)):
            qs, out = strided(q, *pad), strided(torch.zeros_like(q), *pad)
            rf.attention(su.cache, su.batch, qs, out=out)
            assert torch.equal(out, want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = rf.attention(su.cache, su.batch, q)
            got2 = rf.attention(su.cache, su.batch, q, flags=rf.CHAIN)
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(got2, want)


def test_attention_tiles_and_rows_agree_on_one_token_at_a_time():
    """A chunk gives each token what it gets alone (within both paths' bounds)."""
    rng = np.random.default_rng(20)
    su = Setup(rng, [1500], [100], 1, 128, 64)
    assert by_tiles(su, 4)
    q, q64 = randn(rng, (100, 4, 128))
    whole = check_attention(su, q, q64, "float32")
    for t in (0, 31, 63):
        one = rf.KVBatch(i32(su.table), i32([1500 + t]), i32([0, 1]), 1)
        alone = rf.attention(su.cache, one, q[t:t + 1].contiguous())
        assert torch.allclose(alone[0], whole[t], rtol=1e-4, atol=1e-5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("past,new", [(5, 1), (3000, 1), (150, 40), (4000, 40)])
def test_nan_and_infinite_queries_stay_in_their_rows(dtype, past, new):
    """Single tokens and chunks, one part and several."""
    rng = np.random.default_rng([past, new])
    su = Setup(rng, [past], [new], 1, 64, 64)
    q, q64 = randn(rng, (new, 4, 64), dtype)
    clean = check_attention(su, q, q64, dtype)
    q[0, 1, 5] = float("nan")
    q[new - 1, 2, 7] = float("inf")
    out = rf.attention(su.cache, su.batch, q)
    assert torch.isnan(out[0, 1]).all() and torch.isnan(out[new - 1, 2]).all()
    hit = torch.zeros((new, 4), dtype=torch.bool, device="cuda")
    hit[0, 1] = hit[new - 1, 2] = True
    assert torch.equal(out[~hit], clean[~hit])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim,heads,window,past,new", [(64, 8, 1, [500], [600]), (64, 8, 128, [300, 0, 9], [300, 257, 31]),
                                                       (128, 4, 200, [40, 1000], [400, 301])])
def test_attention_long_chunks_under_a_window(dtype, dim, heads, window, past, new):
    rng = np.random.default_rng([dim, window])
    su = Setup(rng, past, new, 1, dim, 64)
    assert by_tiles(su, heads, window)
    q, q64 = randn(rng, (su.n_tok, heads, dim), dtype, 2.0)
    check_attention(su, q, q64, dtype, window=window, sinks=rng.standard_normal(heads).astype(np.float32))
    assert rf.device_status() == rf.OK
