"""The routed FFN of a layer over 16-bit residual streams, and the fp32 outputs
of products with 16-bit inputs that its router needs."""
import numpy as np
import pytest
import torch

import quantized_weight_streaming_dequant_gb300 as rf
from chunk_helpers import DTYPES, FMTS, NAMES, check, moe_reference, randn, raw, reference
from oracle import chunk as oc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_weight_streaming_dequant_gb300 import build
    build.build()
    yield
    assert rf.device_status() == rf.OK


def host(t):
    return t.double().cpu().numpy()


def two_terms(fmt, w, x, **kw):
    """reference() of a product of 16-bit inputs with fp32 outputs: weights as
    two fp16 terms, which is what fp16 calls have; the values of x are exact."""
    return reference(fmt, "float16", w, x, **kw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("n_tok,rows,blocks", [(1, 40, 8), (8, 130, 17), (13, 65, 24), (50, 77, 33), (200, 300, 9), (300, 129, 40), (5, 64, 344)])
def test_fp32_outputs(fmt, dtype, n_tok, rows, blocks):
    in_dim = max(1, blocks // 8) * 256 if fmt == rf.Q4_K else 32 * blocks
    rng = np.random.default_rng([n_tok, rows])
    W, w = raw(fmt, 1, rows, in_dim, 7)
    U, u = raw(fmt, 1, rows, in_dim, 8)
    x, xv = randn(rng, (n_tok, in_dim), dtype)
    b, bv = randn(rng, (rows,), "float32")
    res, resv = randn(rng, (n_tok, rows), "float32")
    through = (lambda *a, **k: reference(fmt, "float32", *a, **k)) if dtype == "float32" else \
        (lambda *a, **k: two_terms(fmt, *a, **k))
    got = rf.gemm_fused(fmt, W, 0, rows, in_dim, x, bias=b, residual=res, y_f32=True)
    y, bound = through(w[0], xv, bias=bv, residual=resv)
    assert got.dtype == torch.float32
    check(got, y, bound, "float32")
    buf = torch.full((n_tok, rows + 3), 7.0, device="cuda")
    out = buf[:, 1:1 + rows]
    rf.gemm_fused(fmt, W, 0, rows, in_dim, x, out, act=rf.ACT_SWIGLU, up=U, y_f32=True,
                  workspace=rf.gemm_fused_workspace(fmt, rows, in_dim, x, y_f32=True))
    y, bound = through(w[0], xv, kind=oc.SWIGLU, up=u[0])
    check(out, y, bound, "float32")
    assert (buf[:, 0] == 7).all() and (buf[:, 1 + rows:] == 7).all()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("sizes", [[3, 0, 1, 8, 2], [40, 0, 17, 200]], ids=str)
def test_grouped_fp32_outputs(fmt, dtype, sizes):
    in_dim, rows, n = 512, 70, len(sizes)
    offsets = np.concatenate([[0], np.cumsum(sizes)])
    rng = np.random.default_rng(n)
    W, w = raw(fmt, n, rows, in_dim, 9)
    x, xv = randn(rng, (int(offsets[-1]), in_dim), dtype)
    at = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    got = rf.gemm_grouped(fmt, W, rows, in_dim, x, at, act=rf.ACT_SILU, y_f32=True,
                          workspace=rf.gemm_grouped_workspace(fmt, n, rows, in_dim, x, x.shape[0], y_f32=True))
    for g in range(n):
        a, e = offsets[g], offsets[g + 1]
        y, bound = two_terms(fmt, w[g], xv[a:e], kind=oc.SILU)
        check(got[a:e], y, bound, "float32", f"group {g}")


def test_a_dtype_of_x_alone_is_for_products():
    """The outputs' type has to be the call's; the routed FFN has no such form."""
    x = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")
    W, _ = raw(rf.Q4_0, 1, 8, 64, 1)
    with pytest.raises(ValueError, match="Y must be"):
        rf.gemm_fused(rf.Q4_0, W, 0, 8, 64, x, torch.zeros((2, 8), device="cuda"))
    with pytest.raises(ValueError, match="Y must be"):
        rf.gemm_fused(rf.Q4_0, W, 0, 8, 64, x, torch.zeros((2, 8), dtype=x.dtype, device="cuda"), y_f32=True)
    with pytest.raises(ValueError, match="residual must be"):
        rf.gemm_fused(rf.Q4_0, W, 0, 8, 64, x, residual=torch.zeros((2, 8), dtype=x.dtype, device="cuda"), y_f32=True)


def layer(rng, E, k, ff, embd, bias):
    G, g = raw(rf.MXFP4, E, ff, embd, 1)
    U, u = raw(rf.MXFP4, E, ff, embd, 2)
    D, d = raw(rf.MXFP4, E, embd, ff, 3)
    R, r = raw(rf.Q8_0, 1, E, embd, 4)
    nw = torch.from_numpy(1 + 0.1 * rng.standard_normal(embd).astype(np.float32)).cuda()
    from quantized_weight_streaming_dequant_gb300.layer import RoutedFFN
    b = torch.from_numpy(bias.astype(np.float32)).cuda()
    return RoutedFFN(rf.MXFP4, E, k, embd, ff, G, U, D, rf.Q8_0, R, nw, router_bias=b), (g, u, d, r[0])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n_tok", [1, 6, 45, 130])
def test_a_layer_of_experts(n_tok, dtype):
    """Logits in fp32 whatever the stream's type, from the normed input as it
    was rounded; large biases, next to which a 16-bit logit keeps little of what
    tells experts apart, so that many would tie."""
    rng = np.random.default_rng([n_tok, 3])
    E, k, ff, embd = 24, 4, 192, 256
    bias = 60.0 + 0.05 * rng.standard_normal(E)
    ffn, (g, u, d, r) = layer(rng, E, k, ff, embd, bias)
    res, resv = randn(rng, (n_tok, embd), dtype, 1.0)
    o = ffn.step(res)
    assert o["logits"].dtype == torch.float32 and o["x"].dtype == o["y"].dtype == res.dtype
    x, bv = host(o["x"]), bias.astype(np.float32).astype(np.float64)
    y, bound = reference(rf.Q8_0, "float32", r, x, bias=bv) if dtype == "float32" else two_terms(rf.Q8_0, r, x, bias=bv)
    check(o["logits"], y, bound, "float32")
    # The experts are those of the 64-bit logits wherever these are told apart.
    lim = bound + 2.0 ** -23 * np.abs(y)
    ranked = -np.sort(-y, axis=1)
    clear = (ranked[:, :k] - ranked[:, 1:k + 1]).min(1) > 2 * lim.max(1)
    assert clear.mean() > 0.9
    idx, *_ = oc.route(host(o["logits"]), k)
    assert np.array_equal(idx[clear], oc.route(y, k)[0][clear])
    y, bound = moe_reference(rf.MXFP4, dtype, host(o["logits"]), k, g, u, d, x, residual=resv)
    check(o["y"], y, bound, dtype)


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("n_tok", [7, 40, 300])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_a_routed_ffn_is_off_by_little_more_than_its_outputs_rounding(fmt, n_tok, dtype):
    """Each rounding inside is an eighth of half a step of the output's type at
    most: h in fp16 calls as two fp16 terms (2^-22 of a value), in bf16 calls to
    fp16 (2^-11 against 2^-8), as their weights of all formats but MXFP4.  Errors
    of that size that fall evenly add 1/8 of the output's own in root mean square
    each, in quadrature: three from up's and down's weights and from h, and one
    from gate's, times z silu'(z) / silu(z) = 1 + z (1 - sigmoid(z)), at most 1.28
    where silu is not small: sqrt(1 + (3 + 1.28^2) / 64), 3.6 % over it; in fp16
    calls nothing that shows."""
    rng = np.random.default_rng([n_tok, 8])
    E, k, ff, embd = 7, 2, 512, 768
    G, g = raw(fmt, E, ff, embd, 1)
    U, u = raw(fmt, E, ff, embd, 2)
    D, d = raw(fmt, E, embd, ff, 3)
    x, xv = randn(rng, (n_tok, embd), dtype)
    logits, lv = randn(rng, (n_tok, E), "float32")
    got = rf.moe_ffn_tokens(fmt, logits, k, G, U, D, ff, embd, x)
    y, b = moe_reference(fmt, dtype, lv, k, g, u, d, xv)
    check(got, y, b, dtype)
    rms = lambda a: float(np.sqrt(np.mean((a / np.abs(y).max(1, keepdims=True)) ** 2)))  # noqa: E731
    own = rms(torch.from_numpy(y).to(x.dtype).double().numpy() - y)
    assert rms(host(got) - y) <= (1.005 if dtype == "float16" else 1.036) * own
