"""The whole decoder layer over the paged cache: every stage against the fp64
oracle on that stage's own inputs, prompts and single tokens."""
import numpy as np
import pytest
import torch

import oracle
import quantized_weight_streaming_dequant_gb300 as rf
import synthetic as syn
from decoder_helpers import i32
from gpu_helpers import derived_gemm_bound, dev_tensor, gemv_tol
from oracle import decoder as od
from quantized_weight_streaming_dequant_gb300.layer import DecoderLayer

pytestmark = pytest.mark.gpu

D, FF, NH, NK, HD, PAGE = 256, 512, 4, 2, 64, 64


def make(fmt, rng, **kw):
    shapes = dict(wq=(NH * HD, D), wk=(NK * HD, D), wv=(NK * HD, D), wo=(D, NH * HD), w_gate=(FF, D), w_up=(FF, D), w_down=(D, FF))
    W = {n: syn.quant_matrix(fmt, r, c, seed=50 + i) for i, (n, (r, c)) in enumerate(shapes.items())}
    norms = {n: (1 + 0.2 * rng.standard_normal(D)).astype(np.float32) for n in ("norm_attn", "norm_ffn", "post_attn", "post_ffn")}
    a = np.arange(512)[:, None] * (10000.0 ** (-np.arange(HD // 2) / (HD // 2)))
    tab = dict(cos=np.cos(a).astype(np.float32), sin=np.sin(a).astype(np.float32))
    sinks = rng.standard_normal(NH).astype(np.float32)
    dev = {n: dev_tensor(v) for n, v in {**W, **norms, **tab}.items()}
    layer = DecoderLayer(fmt, D, FF, NH, NK, HD, sinks=dev_tensor(sinks), **dev, **kw)
    return layer, W, norms, tab


def project_check(fmt, W, rows, cols, x, y):
    """One token and up to eight: the GEMV's parity bound; chunks: the GEMM's."""
    x, y = x.reshape(-1, cols), y.reshape(-1, rows)
    if len(x) > 8 and fmt != rf.Q6_K:
        bound = derived_gemm_bound(fmt, W, 0, rows, cols, x)
        assert (np.abs(y - np.stack([oracle.gemv(fmt, W, 0, rows, cols, r) for r in x])) <= bound).all()
        return
    for xr, yr in zip(x, y):
        assert (np.abs(yr - oracle.gemv(fmt, W, 0, rows, cols, xr)) <= gemv_tol(fmt, W, 0, rows, cols, xr)).all()


@pytest.mark.parametrize("fmt", [rf.Q8_0, rf.Q4_0, rf.MXFP4, rf.Q4_K, rf.Q6_K])
def test_prompt_then_tokens(fmt):
    rng = np.random.default_rng(fmt)
    window = 48 if fmt == rf.Q4_0 else 0
    layer, W, norms, tab = make(fmt, rng, window=window, residual_scale=0.5 if fmt == rf.MXFP4 else 1.0)
    cache = rf.KVCache.empty(8, NK, PAGE, HD)
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(255)                                            # nothing that was there counts
    ref = od.Cache(*(t.cpu().numpy() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
    table = np.array([[5, 2, 7]], np.int32)
    past = 0
    for n_tok, first in ((70, True), (1, False), (5, False), (1, True), (1, False)):
        batch = rf.KVBatch(i32(table), i32([past]), i32([0, n_tok]), n_tok)
        residual = dev_tensor(rng.standard_normal((n_tok, D)).astype(np.float32))
        delta = None if first else dev_tensor(rng.standard_normal((n_tok, D)).astype(np.float32))
        o = layer.step(residual, delta, cache, batch, prev_post=None if first else layer.post_ffn, max_len=past + n_tok)
        got = {k: v.double().cpu().numpy() for k, v in o.items()}
        # norm before attention
        r, x = od.norm_residual(None if first else delta.cpu().numpy(), residual.cpu().numpy(),
                                None if first else norms["post_ffn"], None, layer.residual_scale, norms["norm_attn"], np.float32(1e-5))
        np.testing.assert_allclose(got["in"], r, rtol=1e-5, atol=1e-5)
        np.testing.assert_allclose(got["x"], x, rtol=1e-5, atol=1e-5)
        # projections of the GPU's own x, rotation and append of its own q, k, v
        x32 = o["x"].cpu().numpy()
        project_check(fmt, W["wq"], NH * HD, D, x32, got["q"])
        project_check(fmt, W["wk"], NK * HD, D, x32, got["k"])
        project_check(fmt, W["wv"], NK * HD, D, x32, got["v"])
        turn = lambda a: np.stack([od.rotate(a[t], tab["cos"][past + t], tab["sin"][past + t], False) for t in range(n_tok)])  # noqa: E731
        q = turn(o["q"].cpu().numpy())
        assert np.array_equal(o["q_rot"].cpu().numpy(), q)
        ref.append(table, [past], [0, n_tok], turn(o["k"].cpu().numpy()), o["v"].cpu().numpy())
        assert np.array_equal(cache.k.cpu().numpy(), ref.codes[0]) and np.array_equal(cache.v.cpu().numpy(), ref.codes[1])
        # attention over that cache (its accuracy has tests of its own), O, norm, FFN
        again = rf.attention(cache, batch, o["q_rot"], window=window, sinks=layer.sinks, max_len=past + n_tok)
        assert torch.equal(o["attn"], again) and torch.isfinite(again).all() and again.abs().sum() > 0
        project_check(fmt, W["wo"], D, NH * HD, o["attn"].cpu().numpy(), got["o"])
        r, y = od.norm_residual(got["o"], got["in"], norms["post_attn"], None, layer.residual_scale, norms["norm_ffn"], np.float32(1e-5))
        np.testing.assert_allclose(got["residual"], r, rtol=1e-5, atol=1e-5)
        np.testing.assert_allclose(got["y"], y, rtol=1e-5, atol=1e-5)
        project_check(fmt, W["w_down"], D, FF, o["h"].cpu().numpy(), got["delta"])
        past += n_tok
    end, normed = layer.finish(o["residual"], o["delta"], layer.norm_attn)
    r, y = od.norm_residual(got["delta"], got["residual"], norms["post_ffn"], None, layer.residual_scale, norms["norm_attn"], np.float32(1e-5))
    np.testing.assert_allclose(end.cpu().numpy(), r, rtol=1e-5, atol=1e-5)
    np.testing.assert_allclose(normed.cpu().numpy(), y, rtol=1e-5, atol=1e-5)
    assert rf.device_status() == rf.OK
