"""Products whose persistent CTAs take several pieces of work: phases of the
rings that carry over from one to the next, the second set of sums, item slots
that come round again.  For each tile width of chunk_kernel (32, 64, 128 and
192 operand rows) and of few_kernel (8, 16), each format and type, with at least
two pieces of work for every CTA; and calls whose inputs are shared out in parts
against calls that are not."""
import functools

import numpy as np
import pytest
import torch

import oracle
import quantized_weight_streaming_dequant_gb300 as rf
import synthetic as syn
from chunk_helpers import DTYPES, FMTS, NAMES, TORCH, act_bound, check, moe_reference, product_bound, randn, raw
from oracle import chunk as oc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_weight_streaming_dequant_gb300 import build
    build.build()
    yield
    assert rf.device_status() == rf.OK


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@functools.lru_cache(maxsize=2)
def matrix(fmt, rows, in_dim, seed):
    W = syn.quant_matrix(fmt, rows, in_dim, seed)
    w = np.ascontiguousarray(oracle.dequantize(fmt, W).reshape(rows, in_dim))
    return torch.from_numpy(W).cuda(), torch.from_numpy(w).cuda().double()


def product(fmt, dtype, w, x, bias=None):
    """(z, bound) of x through w (device, fp64), by the bounds of the helpers."""
    a = w.abs()
    z, A = x @ w.T, x.abs() @ a.T
    host = lambda t: t.cpu().numpy()  # noqa: E731
    b = product_bound(fmt, dtype, w.shape[1], host(A), host(a.sum(1))[None], host(x.abs().sum(1))[:, None],
                      host(x.abs().amax(1))[:, None])
    z = host(z)
    if bias is not None:
        z = z + bias
        b = b + 2.0 ** -23 * (np.abs(z) + np.abs(bias))
    return z, b


def inputs(dtype, n_tok, in_dim, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n_tok, in_dim), generator=g, device="cuda").to(TORCH[dtype])
    return x, x.double()


def in_dim_of(fmt, chunks, odd):
    """Inputs of `chunks` raw chunks, the last of them short (not Q4_K's)."""
    if fmt == rf.Q4_K:
        return 256 * chunks
    return (512 if fmt == rf.MXFP4 else 256) * (chunks - 1) + 32 * odd


# (tokens by type, tile's operand rows): one tile, or several whose last is short
WIDTHS = {"float32": [(12, 32), (27, 64), (150, 128)], "float16": [(30, 32), (50, 64), (140, 128)],
          "bfloat16": [(19, 32), (64, 64), (250, 128), (400, 192)]}


@pytest.mark.parametrize("dtype,n_tok,width", [(d, n, w) for d in DTYPES for n, w in WIDTHS[d]])
@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_products_of_several_items_a_cta(fmt, dtype, n_tok, width, gated):
    tiles = -(-n_tok * (2 if dtype == "float32" else 1) // width)
    cols = 64 if gated else 128
    rows = (5 * sms() // 2 // tiles + 1) * cols - 37
    assert tiles * -(-rows // cols) >= 2 * sms()
    in_dim = in_dim_of(fmt, 2, 5)
    W, w = matrix(fmt, rows, in_dim, 3)
    x, xv = inputs(dtype, n_tok, in_dim, n_tok)
    b = torch.randn(rows, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    bv = b.double().cpu().numpy()
    if gated:
        U = W.flip(0).contiguous()
        u = w.flip(0)
        call = lambda: rf.gemm_fused(fmt, W, 0, rows, in_dim, x, act=rf.ACT_SWIGLU, up=U, up_bias=b)  # noqa: E731
        (z, bz), (v, bu) = product(fmt, dtype, w, xv), product(fmt, dtype, u, xv, bv)
        y = oc.act(oc.SWIGLU, z, v)
        bound = act_bound(oc.SWIGLU, z, bz, v, bu, y)
    else:
        call = lambda: rf.gemm_fused(fmt, W, 0, rows, in_dim, x, bias=b)  # noqa: E731
        y, bound = product(fmt, dtype, w, xv, bv)
        bound = act_bound(oc.NONE, y, bound, None, 0.0, y)
    got = call()
    check(got, y, bound, dtype)
    for _ in range(3):
        assert torch.equal(call(), got)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("width", [8, 16])
def test_few_tokens_of_several_items_a_cta(fmt, dtype, width):
    n_tok = (width if dtype != "float32" else width // 2) - 1
    rows = (9 * sms() // 2 + 1) * 128 - 37                 # two CTAs an SM
    in_dim = in_dim_of(fmt, 3, 7)
    W, w = matrix(fmt, rows, in_dim, 4)
    x, xv = inputs(dtype, n_tok, in_dim, width)
    y, bound = product(fmt, dtype, w, xv)
    got = rf.gemm_fused(fmt, W, 0, rows, in_dim, x)
    check(got, y, act_bound(oc.NONE, y, bound, None, 0.0, y), dtype)
    for _ in range(3):
        assert torch.equal(rf.gemm_fused(fmt, W, 0, rows, in_dim, x), got)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("sizes", [[300, 129, 0, 193, 384, 17, 200, 1000], [3, 1, 0, 9, 2, 5, 0, 8, 4, 30, 1, 1]], ids=["large", "few"])
def test_groups_of_several_items_a_cta(fmt, dtype, sizes):
    """Tiles of one group after another's, whole ones and ragged ends (in 16
    bits the first sizes take tiles of 192 rows where one term does)."""
    n, n_row = len(sizes), sum(sizes)
    least = sum(-(-s // 192) for s in sizes) if n_row > 200 else sum(s > 0 for s in sizes)
    rows = ((2 if n_row > 200 else 4) * sms() // least + 2) * 128 - 61
    in_dim = in_dim_of(fmt, 2, 3)
    W, w = matrix(fmt, n * rows, in_dim, 5)
    x, xv = inputs(dtype, n_row, in_dim, 6)
    offsets = np.concatenate([[0], np.cumsum(sizes)])
    at = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    got = rf.gemm_grouped(fmt, W, rows, in_dim, x, at, act=rf.ACT_GELU)
    for g in range(n):
        a, e = offsets[g], offsets[g + 1]
        if a == e:
            continue
        z, b = product(fmt, dtype, w[g * rows:(g + 1) * rows], xv[a:e])
        y = oc.act(oc.GELU, z)
        check(got[a:e], y, act_bound(oc.GELU, z, b, None, 0.0, y), dtype, f"group {g}")
    for _ in range(3):
        assert torch.equal(rf.gemm_grouped(fmt, W, rows, in_dim, x, at, act=rf.ACT_GELU), got)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", [rf.MXFP4, rf.Q4_0], ids=NAMES.get)
def test_a_routed_ffn_of_wide_tiles(fmt, dtype):
    """Few experts with many rows each: tiles of 192 rows in bf16 (and in fp16
    of MXFP4), several pieces of work a CTA in both products."""
    E, k, n_tok, ff, embd = 8, 2, 1001, 1344, 1280
    rng = np.random.default_rng(7)
    G, g = raw(fmt, E, ff, embd, 1)
    U, u = raw(fmt, E, ff, embd, 2)
    D, d = raw(fmt, E, embd, ff, 3)
    x, xv = randn(rng, (n_tok, embd), dtype)
    logits, lv = randn(rng, (n_tok, E), "float32")
    got = rf.moe_ffn_tokens(fmt, logits, k, G, U, D, ff, embd, x)
    y, b = moe_reference(fmt, dtype, lv, k, g, u, d, xv)
    check(got, y, b, dtype)
    for _ in range(3):
        assert torch.equal(rf.moe_ffn_tokens(fmt, logits, k, G, U, D, ff, embd, x), got)


# ------------------------------------------------------------------- parts
def sums_written(space, from_byte, floats):
    """Whether `floats` values behind from_byte of a workspace that was all
    ones have been written (all ones is a NaN, which no sum here is)."""
    return int((space[from_byte:from_byte + 4 * floats].view(torch.int32) != -1).sum()) == floats


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("n_tok", [3, 40])
def test_rows_in_parts_agree_with_whole_rows(fmt, dtype, n_tok, gated):
    """The same 300 rows as a call whose inputs are shared out, which its
    workspace shows, and as the first of a call of so many rows that they are
    not: both within their bound of 64 bits."""
    in_dim, rows, times = 4096, 300, 4 * sms()             # (a segment, so that whole rows need nothing more)
    W, w = matrix(fmt, rows, in_dim, 8)
    U = W.flip(0).contiguous()
    x, xv = inputs(dtype, n_tok, in_dim, 9)
    many = W.repeat(times // 2, 1), U.repeat(times // 2, 1)
    more = {"act": rf.ACT_SWIGLU} if gated else {}
    whole_bytes = rf.gemm_fused_workspace(fmt, many[0].shape[0], in_dim, x).numel()
    space = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
             for n in (rf.gemm_fused_workspace(fmt, rows, in_dim, x).numel(), whole_bytes)]
    # What a call of whole rows needs is the images and what is before them:
    # behind that the parts keep two sums a value at least.
    assert space[0].numel() >= whole_bytes + 4 * 2 * n_tok * rows
    parts = rf.gemm_fused(fmt, W, 0, rows, in_dim, x, up=U if gated else None, workspace=space[0], **more)
    assert sums_written(space[0], whole_bytes, 2 * n_tok * rows)
    whole = rf.gemm_fused(fmt, many[0], 0, many[0].shape[0], in_dim, x, up=many[1] if gated else None, workspace=space[1],
                          **more)[:, :rows]
    z, bz = product(fmt, dtype, w, xv)
    if gated:
        v, bu = product(fmt, dtype, w.flip(0), xv)
        y = oc.act(oc.SWIGLU, z, v)
        b = act_bound(oc.SWIGLU, z, bz, v, bu, y)
    else:
        y, b = z, act_bound(oc.NONE, z, bz, None, 0.0, z)
    check(parts, y, b, dtype, "parts")
    check(whole, y, b, dtype, "whole")
