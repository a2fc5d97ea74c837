"""The chunk operators on the GPU against the fp64 oracle: every format, type
and activation at sizes where tiles, slices, boxes and parts end, ragged and
empty groups, strides, windows, scales at the ends of their range, values that
are not finite, and the calls' other streams, captures and repetitions."""
import numpy as np
import pytest
import torch

import oracle
import quantized_weight_streaming_dequant_gb300 as rf
import synthetic as syn
from chunk_helpers import DTYPES, FMTS, NAMES, TORCH, check, moe_reference, randn, raw, reference
from oracle import chunk as oc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_weight_streaming_dequant_gb300 import build
    build.build()
    yield
    assert rf.device_status() == rf.OK


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def f32(rng, *shape):
    a = rng.standard_normal(shape).astype(np.float32)
    return torch.from_numpy(a).cuda(), a.astype(np.float64)


def inputs(fmt, n):
    """n 32-weight blocks, as the format takes them."""
    return max(1, n // 8) * 256 if fmt == rf.Q4_K else 32 * n


# ------------------------------------------------------------------ routing
ROUTE = [(1, 1, 1), (5, 128, 4), (64, 33, 1), (65, 32, 8), (300, 7, 7), (33, 1024, 8), (2000, 100, 4), (70, 513, 3), (5000, 2, 1)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n_tok,n_expert,k", ROUTE)
def test_route(dtype, n_tok, n_expert, k):
    rng = np.random.default_rng([n_tok, n_expert])
    x = rng.standard_normal((n_tok, n_expert)).astype(np.float32)
    x[rng.random(x.shape) < 0.2] = 0.5                     # ties
    x[rng.random(x.shape) < 0.05] = np.nan
    x[rng.random(x.shape) < 0.05] = -np.inf
    x[rng.random(x.shape) < 0.05] = -0.0
    x[rng.random(x.shape) < 0.05] = 0.0
    x[0] = -np.inf
    wide = torch.full((n_tok, n_expert + 3), 99.0, dtype=TORCH[dtype])
    wide[:, :n_expert] = torch.from_numpy(x).to(TORCH[dtype])
    logits = wide.cuda()[:, :n_expert]                     # strided rows
    r = rf.moe_route_tokens(logits, k)
    idx, w, offsets, order, place = oc.route(wide[:, :n_expert].double().numpy(), k)
    for got, want in ((r.idx, idx), (r.offsets, offsets), (r.order, order), (r.place, place)):
        assert np.array_equal(got.cpu().numpy(), want)
    # exp and the quotient within 2 ulp each, and the sum of k terms
    np.testing.assert_allclose(r.w.cpu().numpy(), w, rtol=(k + 6) * 2.0 ** -24, equal_nan=True)
    if dtype == "float32":                                 # as the single-token router, bit for bit
        for t in range(0, n_tok, max(1, n_tok // 7)):
            i, wt = rf.moe_route(logits[t].contiguous(), k)
            assert torch.equal(i, r.idx[t]) and torch.equal(wt.view(torch.int32), r.w[t].view(torch.int32))


def test_route_of_no_tokens():
    r = rf.moe_route_tokens(torch.zeros((0, 9), device="cuda"), 2)
    assert torch.equal(r.offsets, i32(np.zeros(10))) and r.idx.shape == (0, 2)


# ----------------------------------------------------------- one matrix
# (tokens, rows, 32-weight blocks): a token, ends of granules and tiles, odd
# blocks (rows an odd number of bytes apart for MXFP4), rows behind the last
# super-row, several slices and chunks, parts of the inputs, large tiles
FUSED = [(1, 1, 1), (1, 130, 5), (8, 64, 2), (9, 63, 3), (16, 129, 8), (17, 65, 17), (33, 300, 90), (65, 257, 33), (128, 31, 47),
         (129, 128, 16), (300, 70, 24), (5, 200, 344), (520, 140, 9)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("n_tok,rows,blocks", FUSED)
def test_fused(fmt, dtype, n_tok, rows, blocks):
    in_dim = inputs(fmt, blocks)
    rng = np.random.default_rng([n_tok, rows, blocks])
    kind = [oc.NONE, oc.SILU, oc.GELU, oc.SWIGLU, oc.SWIGLU_CLAMPED][(n_tok + rows + blocks) % 5]
    gated = kind in (oc.SWIGLU, oc.SWIGLU_CLAMPED)
    first = rows % 3                                       # a window that starts inside a super-row
    W, w = raw(fmt, 1, rows + first, in_dim, 11)
    U, u = raw(fmt, 1, rows + first, in_dim, 12) if gated else (None, None)
    x, xv = randn(rng, (n_tok, in_dim), dtype)
    b, bv = f32(rng, rows) if blocks % 2 else (None, None)
    ub, ubv = f32(rng, rows) if gated and rows % 2 else (None, None)
    res, resv = randn(rng, (n_tok, rows), dtype) if n_tok % 2 else (None, None)
    got = rf.gemm_fused(fmt, W, first, rows + first, in_dim, x, act=kind, up=U, bias=b, up_bias=ub, residual=res)
    assert got.dtype == TORCH[dtype]
    y, bound = reference(fmt, dtype, w[0, first:], xv, kind=kind, up=None if u is None else u[0, first:], bias=bv, up_bias=ubv,
                         residual=resv)
    check(got, y, bound, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
def test_fused_strides_alignment_and_in_place_residual(fmt, dtype):
    """Rows of X and Y inside wider buffers, off every 16-byte boundary; the
    residual is Y's own memory; what surrounds it stays as it was."""
    in_dim, rows, n_tok = inputs(fmt, 10), 77, 21
    rng = np.random.default_rng(5)
    W, w = raw(fmt, 1, rows, in_dim, 3)
    x, xv = randn(rng, (n_tok, in_dim), dtype)
    wide = torch.full((n_tok, in_dim + 5), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, 3:3 + in_dim] = x
    y0, y0v = randn(rng, (n_tok, rows), dtype)
    buf = torch.full((n_tok, rows + 9), 7.0, dtype=x.dtype, device="cuda")
    buf[:, 1:1 + rows] = y0
    out = buf[:, 1:1 + rows]
    got = rf.gemm_fused(fmt, W, 0, rows, in_dim, wide[:, 3:3 + in_dim], out, act=rf.ACT_SILU, residual=out)
    assert got.data_ptr() == out.data_ptr()
    y, bound = reference(fmt, dtype, w[0], xv, kind=oc.SILU, residual=y0v)
    check(out, y, bound, dtype)
    assert (buf[:, 0] == 7).all() and (buf[:, 1 + rows:] == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt,scales", [(rf.MXFP4, (-40, -20)), (rf.MXFP4, (-15, -13)), (rf.MXFP4, (8, 12)), (rf.Q4_0, (1e-7, 1e-6)),
                                        (rf.Q4_0, (3.0, 60.0)), (rf.Q8_0, (0.2, 6.0)), (rf.Q8_0, (1e-7, 1e-5)), (rf.Q4_K, (0.05, 0.4))],
                         ids=lambda v: NAMES.get(v, v) if isinstance(v, int) else str(v))
def test_fused_scales_at_the_ends_of_their_range(fmt, scales, dtype):
    """Subnormal fp16 weights and scales, and weights up to some thousands."""
    in_dim, rows, n_tok = inputs(fmt, 8), 40, 9
    rng = np.random.default_rng(8)
    W, w = raw(fmt, 1, rows, in_dim, 31, scale_range=scales)
    x, xv = randn(rng, (n_tok, in_dim), dtype)
    got = rf.gemm_fused(fmt, W, 0, rows, in_dim, x)
    y, bound = reference(fmt, dtype, w[0], xv)
    if dtype == "float16":
        keep = np.abs(y) < 6e4
        got, y, bound = torch.where(torch.from_numpy(keep).cuda(), got, torch.zeros_like(got)), y * keep, bound * keep
    check(got, y, bound, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_fused_rows_of_very_different_sizes(dtype):
    """Each row of X has a scale of its own; zeros, the type's largest and its
    smallest values, and values far below their row's largest."""
    in_dim, rows = 320, 33
    rng = np.random.default_rng(9)
    W, w = raw(rf.MXFP4, 1, rows, in_dim, 2)
    x = rng.standard_normal((7, in_dim))
    info = torch.finfo(TORCH[dtype])
    top = 1e3 if dtype == "float16" else 2.0 ** 100
    x[0] = 0
    x[1] *= top / 8
    x[2] *= float(info.tiny) * 64 if dtype != "float16" else 2.0 ** -12
    x[3, 1:] *= 2.0 ** -20 if dtype != "float16" else 2.0 ** -8
    x[4, ::2] = 0
    x[5] = 1.0
    t = torch.from_numpy(x).to(TORCH[dtype])
    got = rf.gemm_fused(rf.MXFP4, W, 0, rows, in_dim, t.cuda())
    y, bound = reference(rf.MXFP4, dtype, w[0], t.double().numpy())
    if dtype != "float16":      # the smallest outputs are subnormal
        bound = bound + 2.0 ** -149 * (2.0 ** 16 if dtype == "bfloat16" else 1)
    check(got, y, bound, dtype)
    assert (got[0] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_fused_values_that_are_not_finite_stay_in_their_row(dtype, bad):
    in_dim, rows, n_tok = 192, 70, 20
    rng = np.random.default_rng(10)
    W, w = raw(rf.Q4_0, 1, rows, in_dim, 4)
    x, xv = randn(rng, (n_tok, in_dim), dtype)
    x[7, 100] = bad
    got = rf.gemm_fused(rf.Q4_0, W, 0, rows, in_dim, x)
    assert not torch.isfinite(got[7]).any()
    others = [t for t in range(n_tok) if t != 7]
    y, bound = reference(rf.Q4_0, dtype, w[0], xv[others])
    check(got[others], y, bound, dtype)
    U, _ = raw(rf.Q4_0, 1, rows, in_dim, 5)
    gated = rf.gemm_fused(rf.Q4_0, W, 0, rows, in_dim, x, act=rf.ACT_SWIGLU_CLAMPED, up=U)
    assert torch.isfinite(gated[others]).all()
    if bad != bad:
        assert torch.isnan(gated[7]).all()


def test_weights_that_are_not_finite_stay_in_their_row():
    """A NaN scale (E8M0 255) in one row; the blocks behind a row's last one
    are another row's bytes and must not reach it."""
    in_dim, rows, n_tok = 32 * 3, 150, 18
    rng = np.random.default_rng(11)
    Wn = syn.quant_matrix(rf.MXFP4, rows, in_dim, 6).copy()
    Wn[77, 0] = 255
    W, w = torch.from_numpy(Wn).cuda(), oc.weights(rf.MXFP4, Wn, 1, rows, in_dim)[0]
    x, xv = randn(rng, (n_tok, in_dim), "bfloat16")
    got = rf.gemm_fused(rf.MXFP4, W, 0, rows, in_dim, x)
    assert torch.isnan(got[:, 77]).all()
    keep = [r for r in range(rows) if r != 77]
    y, bound = reference(rf.MXFP4, "bfloat16", w[keep], xv)
    check(got[:, keep], y, bound, "bfloat16")


def test_fused_empty_work():
    W, _ = raw(rf.Q4_0, 1, 8, 64, 1)
    assert rf.gemm_fused(rf.Q4_0, W, 0, 8, 64, torch.zeros((0, 64), device="cuda")).shape == (0, 8)
    assert rf.gemm_fused(rf.Q4_0, W, 4, 4, 64, torch.zeros((3, 64), device="cuda")).shape == (3, 0)


# ------------------------------------------------------------- many groups
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("sizes,rows,blocks", [
    ([0, 3, 0, 0, 17, 1, 40, 0], 70, 5), ([16, 16, 15, 33], 130, 18), ([0, 0, 0], 5, 2), ([200, 0, 1], 64, 9),
    ([1] * 30, 129, 3), ([7, 0, 300, 129], 65, 2)], ids=str)
def test_grouped(fmt, dtype, sizes, rows, blocks):
    """Rows gathered through `order`, some X rows twice, groups empty or
    ragged; rows of Y behind the last group stay as they were."""
    in_dim, n, used, spare = inputs(fmt, blocks), len(sizes), sum(sizes), 5
    rng = np.random.default_rng([n, rows])
    W, w = raw(fmt, n, rows, in_dim, 21)
    U, u = raw(fmt, n, rows, in_dim, 22)
    x, xv = randn(rng, (13, in_dim), dtype)
    order = rng.integers(0, 26, used + spare)
    order[used:] = 1 << 20                                 # no rows of X: never looked at
    b, bv = f32(rng, n, rows)
    res, resv = randn(rng, (used + spare, rows), dtype)
    Y = torch.full((used + spare, rows), 5.0, dtype=x.dtype, device="cuda")
    offsets = np.concatenate([[0], np.cumsum(sizes)])
    rf.gemm_grouped(fmt, W, rows, in_dim, x, i32(offsets), i32(order), 2, Y, act=rf.ACT_SWIGLU, up=U, bias=b, residual=res)
    assert (Y[used:] == 5).all()
    for g in range(n):
        a, e = offsets[g], offsets[g + 1]
        y, bound = reference(fmt, dtype, w[g], xv[order[a:e] // 2], kind=oc.SWIGLU, up=u[g], bias=bv[g], residual=resv[a:e])
        check(Y[a:e], y, bound, dtype, f"group {g}")


def test_grouped_without_order_and_rows_before_the_first_group():
    rng = np.random.default_rng(3)
    W, w = raw(rf.Q8_0, 2, 40, 96, 2)
    x, xv = randn(rng, (20, 96), "float32")
    Y = torch.full((20, 40), 3.0, device="cuda")
    rf.gemm_grouped(rf.Q8_0, W, 40, 96, x, i32([4, 10, 18]), Y=Y)
    assert (Y[:4] == 3).all() and (Y[18:] == 3).all()
    for g, (a, e) in enumerate(((4, 10), (10, 18))):
        y, bound = reference(rf.Q8_0, "float32", w[g], xv[a:e])
        check(Y[a:e], y, bound, "float32")


def test_grouped_bad_offsets_and_rows_are_reported():
    """A group out of order or out of range is skipped, an entry that leaves X
    counts as zeros; the other groups are right."""
    rng = np.random.default_rng(4)
    W, w = raw(rf.Q4_0, 3, 40, 64, 2)
    x, xv = randn(rng, (12, 64), "float32")
    assert rf.device_status() == rf.OK
    for offsets, good in (([0, 5, 3, 12], {0: (0, 5)}), ([-1, 4, 9, 12], {1: (4, 9), 2: (9, 12)}), ([0, 4, 9, 13], {0: (0, 4), 1: (4, 9)})):
        Y = torch.zeros((12, 40), device="cuda")
        rf.gemm_grouped(rf.Q4_0, W, 40, 64, x, i32(offsets), Y=Y)
        assert rf.device_status() == 1
        for g, (a, e) in good.items():
            if offsets == [0, 5, 3, 12] and g == 0:
                e = 3                                      # rows 3, 4 belong to group 2 as well
            y, bound = reference(rf.Q4_0, "float32", w[g], xv[a:e])
            check(Y[a:e], y, bound, "float32", f"{offsets} group {g}")
    for order in ([0, 1, 12, 3], [0, 1, -1, 3], [0, 1, 2 ** 31 - 1, 3]):
        got = rf.gemm_grouped(rf.Q4_0, W, 40, 64, x, i32([0, 4, 4, 4]), i32(order))
        assert rf.device_status() == 1
        y, bound = reference(rf.Q4_0, "float32", w[0], xv[[0, 1, 3]])
        check(got[[0, 1, 3]], y, bound, "float32")
        assert (got[2] == 0).all()
    assert rf.device_status() == rf.OK


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offsets", [[0, 90, 10, 100], [0, 4, 0, 4, 0, 4, 0, 60], [0, 100, 0, 100, 0, 100], [8, 40, 3, 100, 99, 100]], ids=str)
def test_grouped_offsets_that_make_groups_overlap(offsets, dtype):
    """Reported, nothing outside Y's rows is written, and the next call is right."""
    n, n_row, rows, in_dim = len(offsets) - 1, 100, 70, 96
    rng = np.random.default_rng(5)
    W, w = raw(rf.MXFP4, n, rows, in_dim, 2)
    x, xv = randn(rng, (n_row, in_dim), dtype)
    buf = torch.full((n_row + 20, rows), 3.0, dtype=x.dtype, device="cuda")
    need = rf.gemm_grouped_workspace(rf.MXFP4, n, rows, in_dim, x, n_row).numel()
    space = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    rf.gemm_grouped(rf.MXFP4, W, rows, in_dim, x, i32(offsets), Y=buf[10:10 + n_row], workspace=space[:need])
    assert rf.device_status() == 1
    assert (buf[:10] == 3).all() and (buf[10 + n_row:] == 3).all() and (space[need:] == 0x5A).all()
    got = rf.gemm_grouped(rf.MXFP4, W, rows, in_dim, x, i32([0] * n + [n_row]))
    y, bound = reference(rf.MXFP4, dtype, w[n - 1], xv)
    check(got, y, bound, dtype)


@pytest.mark.parametrize("n_group", [1000, 3000])
def test_grouped_many_groups(n_group):
    rng = np.random.default_rng(6)
    sizes = rng.integers(0, 3, n_group)
    offsets = np.concatenate([[0], np.cumsum(sizes)])
    W, w = raw(rf.MXFP4, n_group, 9, 64, 2)
    x, xv = randn(rng, (int(offsets[-1]), 64), "bfloat16")
    got = rf.gemm_grouped(rf.MXFP4, W, 9, 64, x, i32(offsets))
    group = np.repeat(np.arange(n_group), sizes)
    y = np.einsum("ni,nri->nr", xv, w[group])
    A = np.einsum("ni,nri->nr", np.abs(xv), np.abs(w[group]))
    from chunk_helpers import product_bound
    check(got, y, product_bound(rf.MXFP4, "bfloat16", 64, A, np.abs(w[group]).sum(2), np.abs(xv).sum(1)[:, None],
                                np.abs(xv).max(1)[:, None]), "bfloat16")


# ---------------------------------------------------------------- routed FFN
MOE = [(1, 8, 2, 3, 2), (6, 40, 4, 9, 5), (50, 5, 2, 18, 11), (37, 12, 8, 2, 3), (200, 3, 1, 5, 4), (2, 3, 3, 90, 44), (90, 2, 2, 4, 16)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("n_tok,n_expert,k,ff,embd", MOE)
def test_moe(fmt, dtype, n_tok, n_expert, k, ff, embd):
    ff, embd = inputs(fmt, ff), inputs(fmt, embd)
    rng = np.random.default_rng([n_tok, n_expert])
    G, g = raw(fmt, n_expert, ff, embd, 41)
    U, u = raw(fmt, n_expert, ff, embd, 42)
    D, d = raw(fmt, n_expert, embd, ff, 43)
    x, xv = randn(rng, (n_tok, embd), dtype)
    logits, lv = randn(rng, (n_tok, n_expert), DTYPES[n_tok % 3])
    clamped = k % 2 == 0
    more, ref = {}, {}
    if clamped:
        more, ref = {"alpha": 1.702, "limit": 7.0}, {"kind": oc.SWIGLU_CLAMPED}
        for key, shape in (("gate_bias", (n_expert, ff)), ("up_bias", (n_expert, ff)), ("down_bias", (n_expert, embd))):
            more[key], ref[key] = f32(rng, *shape)
    if n_tok % 2:
        more["residual"], ref["residual"] = randn(rng, (n_tok, embd), dtype)
    got = rf.moe_ffn_tokens(fmt, logits, k, G, U, D, ff, embd, x, **more)
    y, bound = moe_reference(fmt, dtype, lv, k, g, u, d, xv, **ref)
    check(got, y, bound, dtype)


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
def test_moe_of_one_token_agrees_with_the_decode_path(fmt):
    """rf_moe_ffn keeps activations in 16 bits, 2^-15 of each block's largest:
    both lie within the parity bar of the routed FFN."""
    E, ff, embd, k = 9, inputs(fmt, 8), inputs(fmt, 16), 2
    Gn, Un, Dn = (syn.stacked_experts(fmt, E, r, c, s) for r, c, s in ((ff, embd, 1), (ff, embd, 2), (embd, ff, 3)))
    x, logits = syn.normal_f32(embd, 4), syn.router_logits(E, 5)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    got = rf.moe_ffn_tokens(fmt, t(logits)[None], k, t(Gn), t(Un), t(Dn), ff, embd, t(x)[None])[0]
    y, _ = rf.moe_ffn(fmt, t(logits), k, t(Gn), t(Un), t(Dn), ff, embd, 0, t(x))
    want, *_ = oracle.moe_ffn(fmt, logits, k, Gn, Un, Dn, ff, embd, x)
    scale = np.abs(want).max()
    assert np.abs(got.cpu().numpy() - want).max() <= 1e-5 * scale
    assert np.abs(y.cpu().numpy() - want).max() <= 2e-3 * scale


def test_moe_in_place_residual_and_strides():
    rng = np.random.default_rng(12)
    E, k, ff, embd, n_tok = 6, 2, 96, 160, 11
    G, g = raw(rf.MXFP4, E, ff, embd, 1)
    U, u = raw(rf.MXFP4, E, ff, embd, 2)
    D, d = raw(rf.MXFP4, E, embd, ff, 3)
    x, xv = randn(rng, (n_tok, embd), "bfloat16")
    logits, lv = randn(rng, (n_tok, E), "float32")
    buf, bv = randn(rng, (n_tok, embd + 3), "bfloat16")
    before = buf.clone()
    out = buf[:, 1:1 + embd]
    rf.moe_ffn_tokens(rf.MXFP4, logits, k, G, U, D, ff, embd, x, out, residual=out)
    y, bound = moe_reference(rf.MXFP4, "bfloat16", lv, k, g, u, d, xv, residual=bv[:, 1:1 + embd])
    check(out, y, bound, "bfloat16")
    assert torch.equal(buf[:, 0], before[:, 0]) and torch.equal(buf[:, 1 + embd:], before[:, 1 + embd:])


# ------------------------------------------------ repeated, captured, elsewhere
def moe_setup(seed=0, n_tok=70, dtype="bfloat16"):
    rng = np.random.default_rng(seed)
    E, k, ff, embd = 12, 4, 288, 320
    G, _ = raw(rf.MXFP4, E, ff, embd, 1)
    U, _ = raw(rf.MXFP4, E, ff, embd, 2)
    D, _ = raw(rf.MXFP4, E, embd, ff, 3)
    x, _ = randn(rng, (n_tok, embd), dtype)
    logits, _ = randn(rng, (n_tok, E), "float32")
    return (G, U, D, ff, embd), logits, x, k


def test_repeated_calls_give_the_same_bits_and_share_a_workspace():
    w, logits, x, k = moe_setup()
    ws = rf.moe_tokens_workspace(rf.MXFP4, logits.shape[1], k, w[3], w[4], x)
    first = rf.moe_ffn_tokens(rf.MXFP4, logits, k, *w, x, workspace=ws)
    for _ in range(5):
        ws.fill_(255)                                      # nothing of it has to survive, or to start at zero
        other = rf.moe_ffn_tokens(rf.MXFP4, logits.flip(0).contiguous(), k, *w, x, workspace=ws)
        again = rf.moe_ffn_tokens(rf.MXFP4, logits, k, *w, x, workspace=ws)
        assert torch.equal(first, again) and not torch.equal(first, other)


def test_captured_call_follows_its_inputs():
    """A captured routed FFN and a captured grouped product, replayed with other
    logits, offsets and activations."""
    w, logits, x, k = moe_setup()
    _, logits2, x2, _ = moe_setup(1)
    want = [rf.moe_ffn_tokens(rf.MXFP4, a, k, *w, b).clone() for a, b in ((logits, x), (logits2, x2))]
    W, _ = raw(rf.Q4_0, 3, 50, 64, 9)
    xs, _ = randn(np.random.default_rng(1), (30, 64), "float32")
    offs = [i32([0, 7, 7, 30]), i32([0, 0, 20, 25])]
    Yw = []
    for o in offs:
        Y = torch.zeros((30, 50), device="cuda")
        Yw.append(rf.gemm_grouped(rf.Q4_0, W, 50, 64, xs, o, Y=Y))
    la, xa, oa = logits.clone(), x.clone(), offs[0].clone()
    ws = rf.moe_tokens_workspace(rf.MXFP4, logits.shape[1], k, w[3], w[4], x)
    ws2 = rf.gemm_grouped_workspace(rf.Q4_0, 3, 50, 64, xs, 30)
    out, Y = torch.empty_like(x), torch.zeros((30, 50), device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rf.moe_ffn_tokens(rf.MXFP4, la, k, *w, xa, out, workspace=ws)
        Y.zero_()
        rf.gemm_grouped(rf.Q4_0, W, 50, 64, xs, oa, Y=Y, workspace=ws2)
    for i, (a, b) in enumerate(((logits, x), (logits2, x2), (logits, x))):
        la.copy_(a), xa.copy_(b), oa.copy_(offs[i % 2])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i % 2]) and torch.equal(Y, Yw[i % 2])


def test_two_calls_on_two_streams():
    w, logits, x, k = moe_setup(2, 150)
    _, logits2, x2, _ = moe_setup(3, 150)
    want = [rf.moe_ffn_tokens(rf.MXFP4, a, k, *w, b) for a, b in ((logits, x), (logits2, x2))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [rf.moe_ffn_tokens(rf.MXFP4, a, k, *w, b, stream=s) for (a, b), s in zip(((logits, x), (logits2, x2)), streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_results_do_not_depend_on_other_rows():
    """A token's values are the same bits whatever the other tokens hold."""
    W, _ = raw(rf.Q4_K, 1, 100, 512, 5)
    x, _ = randn(np.random.default_rng(2), (40, 512), "float16")
    a = rf.gemm_fused(rf.Q4_K, W, 0, 100, 512, x)
    x2 = x.clone()
    x2[:13], x2[14:] = 100, float("inf")
    b = rf.gemm_fused(rf.Q4_K, W, 0, 100, 512, x2)
    assert torch.equal(a[13], b[13])


def test_parts_agree_with_whole_rows():
    """The same rows as part of a call whose inputs are shared out, and of one
    whose are not."""
    fmt, in_dim, rows = rf.Q4_0, 11008, 300
    W, w = raw(fmt, 1, rows, in_dim, 5)
    x, xv = randn(np.random.default_rng(3), (3, in_dim), "float32")
    y, bound = reference(fmt, "float32", w[0], xv)
    check(rf.gemm_fused(fmt, W, 0, rows, in_dim, x), y, bound, "float32")


def test_a_withheld_copy_ends_the_launch_and_the_device_recovers():
    """One slice's activations are never copied: the product gives up after 1
    ms, every role stops, and the next calls give the bits of the call before."""
    import time
    for fmt, n_tok, in_dim in ((rf.Q4_0, 70, 1024), (rf.MXFP4, 300, 2880)):
        W, _ = raw(fmt, 1, 384, in_dim, 1)
        for dtype in DTYPES:
            x, _ = randn(np.random.default_rng(1), (n_tok, in_dim), dtype)
            want = rf.gemm_fused(fmt, W, 0, 384, in_dim, x)
            assert rf.device_status() == rf.OK
            rf.debug_arm_wait_fault(1000)
            t0 = time.perf_counter()
            rf.gemm_fused(fmt, W, 0, 384, in_dim, x)
            assert rf.device_status() == 6
            assert time.perf_counter() - t0 < 1.0
            assert rf.device_status() == rf.OK
            for _ in range(2):
                assert torch.equal(rf.gemm_fused(fmt, W, 0, 384, in_dim, x), want)
    assert rf.device_status() == rf.OK


# ------------------------------------------- few rows a group, and one more
# (4 fp32 and 8 16-bit tokens share eight columns of a product, 8 and 16 take
# tiles of their own, 9 and 17 the way through tensor memory)
FEW = [1, 4, 5, 8, 9, 16, 17]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n_tok", FEW)
@pytest.mark.parametrize("fmt,scales", [(rf.MXFP4, (-40, -20)), (rf.MXFP4, (-15, -13)), (rf.MXFP4, (8, 12)), (rf.Q4_0, (1e-7, 1e-6)),
                                        (rf.Q8_0, (1e-7, 1e-5)), (rf.Q8_0, (0.2, 6.0)), (rf.Q4_K, (0.05, 0.4))],
                         ids=lambda v: NAMES.get(v, v) if isinstance(v, int) else str(v))
def test_few_tokens_scales_at_the_ends_of_their_range(fmt, scales, n_tok, dtype):
    in_dim, rows = inputs(fmt, 24), 70
    rng = np.random.default_rng(n_tok)
    W, w = raw(fmt, 1, rows, in_dim, 33, scale_range=scales)
    x, xv = randn(rng, (n_tok, in_dim), dtype)
    got = rf.gemm_fused(fmt, W, 0, rows, in_dim, x)
    y, bound = reference(fmt, dtype, w[0], xv)
    if dtype == "float16":
        keep = np.abs(y) < 6e4
        got, y, bound = torch.where(torch.from_numpy(keep).cuda(), got, torch.zeros_like(got)), y * keep, bound * keep
    check(got, y, bound, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
def test_few_tokens_in_many_groups(fmt, dtype):
    """Most groups empty, some with more rows than a tile has; blocks that end
    inside four slices; rows behind the last super-row; Y's tail as it was."""
    sizes = [0] * 30 + [1, 23, 0, 5, 4, 9, 17] + [0] * 20 + [2]
    in_dim, rows, n = inputs(fmt, 27), 77, len(sizes)
    used = sum(sizes)
    rng = np.random.default_rng(6)
    W, w = raw(fmt, n, rows, in_dim, 23)
    x, xv = randn(rng, (used, in_dim), dtype)
    b, bv = f32(rng, n, rows)
    offsets = np.concatenate([[0], np.cumsum(sizes)])
    Y = torch.full((used + 3, rows), 4.0, dtype=x.dtype, device="cuda")
    rf.gemm_grouped(fmt, W, rows, in_dim, torch.cat([x, x[:3]]), i32(offsets), Y=Y, act=rf.ACT_SILU, bias=b)
    assert (Y[used:] == 4).all()
    for g in np.flatnonzero(sizes):
        a, e = offsets[g], offsets[g + 1]
        y, bound = reference(fmt, dtype, w[g], xv[a:e], kind=oc.SILU, bias=bv[g])
        check(Y[a:e], y, bound, dtype, f"group {g}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n_tok", [4, 8, 16])
def test_few_tokens_not_finite_stay_in_their_row(n_tok, dtype):
    """NaN and infinities of one token, and a weight row of NaN scales whose
    blocks lie behind the row before it."""
    in_dim, rows = 32 * 5, 90
    rng = np.random.default_rng(12)
    Wn = syn.quant_matrix(rf.MXFP4, rows, in_dim, 8).copy()
    Wn[50, ::17] = 255
    W, w = torch.from_numpy(Wn).cuda(), oc.weights(rf.MXFP4, Wn, 1, rows, in_dim)[0]
    keep = [r for r in range(rows) if r != 50]
    for bad in (float("nan"), float("inf")):
        x, xv = randn(rng, (n_tok, in_dim), dtype)
        x[1, 33] = bad
        got = rf.gemm_fused(rf.MXFP4, W, 0, rows, in_dim, x)
        assert torch.isnan(got[:, 50]).all() and not torch.isfinite(got[1]).any()
        others = [t for t in range(n_tok) if t != 1]
        y, bound = reference(rf.MXFP4, dtype, w[keep], xv[others])
        check(got[others][:, keep], y, bound, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_few_tokens_do_not_depend_on_other_rows(dtype):
    for fmt in FMTS:
        W, _ = raw(fmt, 1, 100, 512, 5)
        for n_tok in (4, 8, 16):
            x, _ = randn(np.random.default_rng(2), (n_tok, 512), dtype)
            a = rf.gemm_fused(fmt, W, 0, 100, 512, x)
            x2 = x.clone()
            x2[:2], x2[3:] = 100, float("inf")
            assert torch.equal(a[2], rf.gemm_fused(fmt, W, 0, 100, 512, x2)[2])


def test_a_withheld_copy_of_few_tokens_ends_the_launch():
    import time
    for fmt, in_dim in ((rf.Q8_0, 64), (rf.MXFP4, 2880)):
        W, _ = raw(fmt, 1, 384, in_dim, 1)
        for dtype in DTYPES:
            x, _ = randn(np.random.default_rng(1), (4, in_dim), dtype)
            want = rf.gemm_fused(fmt, W, 0, 384, in_dim, x)
            assert rf.device_status() == rf.OK
            rf.debug_arm_wait_fault(1000)
            t0 = time.perf_counter()
            rf.gemm_fused(fmt, W, 0, 384, in_dim, x)
            assert rf.device_status() == 6
            assert time.perf_counter() - t0 < 1.0
            assert rf.device_status() == rf.OK
            for _ in range(2):
                assert torch.equal(rf.gemm_fused(fmt, W, 0, 384, in_dim, x), want)
    assert rf.device_status() == rf.OK


def test_a_layer_of_experts_as_it_is_used():
    """Norm, router, routed FFN with the residual, next norm: the run of a layer
    over a chunk, each step against 64 bits on the values it was given."""
    from oracle import decoder as od
    rng = np.random.default_rng(14)
    E, k, ff, embd, n_tok = 10, 4, 192, 256, 45
    G, g = raw(rf.MXFP4, E, ff, embd, 1)
    U, u = raw(rf.MXFP4, E, ff, embd, 2)
    D, d = raw(rf.MXFP4, E, embd, ff, 3)
    R, r = raw(rf.Q8_0, 1, E, embd, 4)
    b, bv = f32(rng, E)
    res, resv = randn(rng, (n_tok, embd), "float32")
    nw = torch.from_numpy(1 + 0.1 * rng.standard_normal(embd).astype(np.float32)).cuda()
    from quantized_weight_streaming_dequant_gb300.layer import RoutedFFN
    layer = RoutedFFN(rf.MXFP4, E, k, embd, ff, G, U, D, rf.Q8_0, R, nw, router_bias=b)
    o = layer.step(res)
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    _, x = od.norm_residual(None, resv, None, None, 1.0, host(nw), layer.eps)
    np.testing.assert_allclose(host(o["x"]), x, rtol=1e-5, atol=1e-6)
    y, bound = reference(rf.Q8_0, "float32", r[0], host(o["x"]), bias=bv)
    check(o["logits"], y, bound, "float32")
    y, bound = moe_reference(rf.MXFP4, "float32", host(o["logits"]), k, g, u, d, host(o["x"]), residual=resv)
    check(o["y"], y, bound, "float32")
    one = layer.step(res[:1])
    check(one["y"], y[:1], bound[:1] + 1e-6 * np.abs(y[:1]).max(), "float32")
