"""Products of very long rows.  The tensor cores truncate their additions, and
on a sum of one sign that adds up; so a sum leaves them for a rounded addition
after a bounded number of inputs, however long the row is."""
import numpy as np
import pytest
import torch

import oracle
import quantized_weight_streaming_dequant_gb300 as rf
import synthetic as syn
from chunk_helpers import DTYPES, FMTS, NAMES, TORCH

pytestmark = pytest.mark.gpu

# Inputs of a sum within the tensor cores at most, as the header states them,
# and products of sixteen inputs by terms of the weights.
def steps(fmt, dtype, y_f32):
    if dtype == "float32":
        return 16
    two = fmt != rf.MXFP4 and (y_f32 or dtype == "float16")
    return (4096 if y_f32 or dtype == "float16" else 16384) // 16 * (2 if two else 1)


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_weight_streaming_dequant_gb300 import build
    build.build()
    yield
    assert rf.device_status() == rf.OK


def matrix(fmt, rows, in_dim, seed):
    W = syn.quant_matrix(fmt, rows, in_dim, seed)
    w = oracle.dequantize(fmt, W).reshape(rows, in_dim)
    return torch.from_numpy(W).cuda(), torch.from_numpy(np.ascontiguousarray(w)).cuda().double()


def one_sign(w, n_tok, dtype):
    """Inputs whose products with w's row 0 are all positive, in sizes that differ."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.rand((n_tok, w.shape[1]), generator=g, device="cuda") + 0.5
    return (x * torch.sign(w[0]).float()).to(TORCH[dtype])


def bound(fmt, dtype, w, x, y_f32=True):
    """As the header states the roundings, before Y's own."""
    x, a = x.double(), w.abs()
    n, exact = w.shape[1], fmt == rf.MXFP4
    rel = 2.0 ** -22 if dtype == "float32" else 0.0
    if not exact:
        rel += 2.0 ** -21 if dtype == "float32" else 2.0 ** -22 if y_f32 or dtype == "float16" else 2.0 ** -11
    # a segment's additions, the rounded ones after each segment (of 128 inputs
    # at least in fp32, 256 in 16 bits), the parts' and the epilogue's
    rel += (steps(fmt, dtype, y_f32) + 1) * 2.0 ** -22 + (n / (128 if dtype == "float32" else 256) + 32) * 2.0 ** -24
    y = x @ w.T
    low = x.abs().sum(1, keepdim=True) * 2.0 ** -25 + a.sum(1)[None] * x.abs().amax(1, keepdim=True) * 2.0 ** -39
    return y, (x.abs() @ a.T) * rel + low


def compare(got, fmt, dtype, w, x, y_f32):
    """got: rows of w over and over, for the tokens x."""
    y, lim = bound(fmt, dtype, w, x, y_f32)
    lim = lim + torch.finfo(got.dtype).eps / 2 * (y.abs() + lim) + (2.0 ** -25 if got.dtype == torch.float16 else 0)
    got = got.double().view(x.shape[0], -1, w.shape[0])
    # what is beyond the type's largest value rounds to infinity (65,504 in fp16)
    over = y.abs() + lim > torch.finfo(torch.float16).max if not y_f32 and dtype == "float16" else torch.zeros_like(y, dtype=torch.bool)
    off = torch.where(over[:, None], 0.0, got - y[:, None]).abs().amax(1)
    assert (off <= lim).all(), f"worst {float((off / lim).max()):.3g} of its bound, {float((off / y.abs())[:, 0].max()):.3g} of the sum"
    assert ((got * y.sign()[:, None])[over[:, None].expand_as(got)] > 6e4).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("n_tok,in_dim", [(40, 1 << 20), (130, 1 << 18), (300, 1 << 18), (300, 16384 + 768), (70, 8192 + 256),
                                          (200, 3 * 16384 + 512)])
def test_sums_shared_out_in_parts(fmt, dtype, n_tok, in_dim):
    W, w = matrix(fmt, 3, in_dim, 3)
    x = one_sign(w, n_tok, dtype)
    for y_f32 in (True, False):
        compare(rf.gemm_fused(fmt, W, 0, 3, in_dim, x, y_f32=y_f32), fmt, dtype, w, x, y_f32)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("n_tok,rows,in_dim", [(4096, 2304, 1 << 18), (4096, 2304, 3 * 16384 + 512), (2048, 5000, 4096 + 256),
                                               (100, 77824, 8192 + 256), (3, 77824, 1 << 16), (8, 77824, 1 << 16),
                                               (16, 77824, 1 << 16)])
def test_sums_of_whole_rows(fmt, dtype, n_tok, rows, in_dim):
    """Calls of so many pieces that none is shared out (the sixteen tokens and
    four rows that are compared come again and again)."""
    W, w = matrix(fmt, 4, in_dim, 3)
    x = one_sign(w, 16, dtype)
    many = x.repeat((n_tok + 15) // 16, 1)[:n_tok]
    stack = W.view(4, -1).repeat(rows // 4, 1)
    for y_f32 in (True, False):
        got = rf.gemm_fused(fmt, stack, 0, rows, in_dim, many, y_f32=y_f32)
        n = min(n_tok, 16)
        compare(got[:n], fmt, dtype, w, x[:n], y_f32)
        if n_tok > 16:
            assert torch.equal(got[n_tok // 16 * 16 - 16:n_tok // 16 * 16], got[:16])


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_long_rows_of_many_items(dtype):
    """More pieces of work than SMs, each of several segments; gated, in groups,
    with a bias; and the same bits when the call is repeated or replayed."""
    fmt, in_dim, rows, n = rf.Q8_0, 3 * 8192 + 64, 1100, 3
    W, w = matrix(fmt, n * rows, in_dim, 4)
    U, u = matrix(fmt, n * rows, in_dim, 5)
    sizes = [300, 1, 555]
    offsets = np.concatenate([[0], np.cumsum(sizes)])
    at = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    x = torch.randn((int(offsets[-1]), in_dim), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(TORCH[dtype])
    b = torch.randn((n, rows), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    ws = rf.gemm_grouped_workspace(fmt, n, rows, in_dim, x, x.shape[0], y_f32=True)
    call = lambda out=None: rf.gemm_grouped(fmt, W, rows, in_dim, x, at, Y=out, act=rf.ACT_SWIGLU, up=U, bias=b,  # noqa: E731
                                            workspace=ws, y_f32=True)
    got = call()
    for g in range(n):
        a, e = offsets[g], offsets[g + 1]
        z, bz = bound(fmt, dtype, w[g * rows:(g + 1) * rows], x[a:e])
        v, bv = bound(fmt, dtype, u[g * rows:(g + 1) * rows], x[a:e])
        z = z + b[g].double()
        f = z * torch.sigmoid(z)
        # |silu'| <= 1.1, and 2^-20 for the activation's arithmetic
        lim = f.abs() * bv + 1.1 * (v.abs() + bv) * (bz + 2.0 ** -23 * z.abs()) + 2.0 ** -20 * (f * v).abs() + 1e-30
        off = (got[a:e].double() - f * v).abs()
        assert (off <= lim).all(), f"group {g}: worst {float((off / lim).max()):.3g} of its bound"
    for _ in range(3):
        ws.fill_(255)
        assert torch.equal(call(), got)
    out = torch.empty_like(got)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, got)


def test_a_long_down_projection_of_a_routed_ffn():
    """Long rows inside the routed FFN: its second product's inputs."""
    from chunk_helpers import check, moe_reference, randn, raw
    rng = np.random.default_rng(6)
    E, k, ff, embd = 3, 2, 8192 * 2 + 512, 64
    G, g = raw(rf.Q4_0, E, ff, embd, 1)
    U, u = raw(rf.Q4_0, E, ff, embd, 2)
    D, d = raw(rf.Q4_0, E, embd, ff, 3)
    for dtype in ("float16", "bfloat16"):
        for n_tok in (9, 150):
            x, xv = randn(rng, (n_tok, embd), dtype)
            logits, lv = randn(rng, (n_tok, E), "float32")
            got = rf.moe_ffn_tokens(rf.Q4_0, logits, k, G, U, D, ff, embd, x)
            y, b = moe_reference(rf.Q4_0, dtype, lv, k, g, u, d, xv)
            check(got, y, b, dtype)
