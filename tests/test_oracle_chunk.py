"""Pins of the chunk oracle by brute force, closed forms and the single-token
oracle -- no GPU -- and of the tests' bounds."""
import math

import numpy as np
import pytest

import oracle
import synthetic as syn
from oracle import chunk as oc


def test_route_matches_the_single_token_router():
    rng = np.random.default_rng(1)
    logits = rng.integers(-3, 4, (40, 11)).astype(np.float32)        # many ties
    logits[3, 4], logits[5], logits[6, 2] = np.nan, -np.inf, -np.inf
    idx, w, offsets, order, place = oc.route(logits, 4)
    for t in range(40):
        i, wt = oracle.router_topk(logits[t], 4)
        assert list(idx[t]) == list(i)
        if t != 5:
            np.testing.assert_allclose(w[t], wt, rtol=1e-6)
    assert offsets[0] == 0 and offsets[-1] == 160 and list(order[place]) == list(range(160))
    experts = idx.ravel()[order]
    assert (np.diff(experts) >= 0).all()
    for e in range(11):
        rows = order[offsets[e]:offsets[e + 1]]
        assert (idx.ravel()[rows] == e).all() and (np.diff(rows) > 0).all()


@pytest.mark.parametrize("kind,ref", [(oc.SILU, oracle.silu), (oc.GELU, oracle.gelu)])
def test_activations(kind, ref):
    z = np.linspace(-30, 30, 41)
    # the scalar GELU is z / 2 (1 + erf): its sum loses up to 2^-53, times |z| / 2 = 15
    np.testing.assert_allclose(oc.act(kind, z), [ref(float(v)) for v in z], rtol=1e-12,
                               atol=15 * 2.0 ** -52 if kind == oc.GELU else 0)


def test_gated_activations():
    z, u = np.array([-9.0, -1.0, 0.5, 3.0, 50.0]), np.array([9.0, -9.0, 0.25, -2.0, 7.5])
    np.testing.assert_allclose(oc.act(oc.SWIGLU, z, u), [oracle.silu(a) * b for a, b in zip(z, u)], rtol=1e-12)
    np.testing.assert_allclose(oc.act(oc.SWIGLU_CLAMPED, z, u, 1.702, 7.0),
                               [oracle.swiglu_clamped(a, b, 1.702, 7.0) for a, b in zip(z, u)], rtol=1e-12)
    assert oc.act(oc.NONE, z) is z


@pytest.mark.parametrize("fmt,in_dim", [(syn.MXFP4, 96), (syn.Q4_0, 64), (syn.Q8_0, 32), (syn.Q4_K, 256)])
def test_product_matches_the_gemv(fmt, in_dim):
    W = syn.quant_matrix(fmt, 6, in_dim, 3)
    x = syn.normal_f32(in_dim, 4)
    z, A, W1, X1 = oc.product(oc.weights(fmt, W, 2, 3, in_dim)[1], x[None])
    np.testing.assert_allclose(z[0], oracle.gemv(fmt, W, 3, 6, in_dim, x), rtol=1e-12)
    assert (A[0] >= np.abs(z[0]) * (1 - 1e-12)).all()
    assert math.isclose(X1[0, 0], np.abs(x.astype(np.float64)).sum())


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("fmt", [syn.MXFP4, syn.Q4_0])
def test_bounds_see_a_lost_block(fmt, dtype):
    """Of 2,880 inputs, one 32-weight block left out, or one slice's rows
    exchanged, is outside every bound."""
    torch = pytest.importorskip("torch")
    from chunk_helpers import TORCH, reference, rounded
    rng = np.random.default_rng(7)
    w = oc.weights(fmt, syn.quant_matrix(fmt, 24, 2880, 5), 1, 24, 2880)[0]
    x = torch.from_numpy(rng.standard_normal((6, 2880)).astype(np.float32)).to(TORCH[dtype]).double().numpy()
    y, b = reference(fmt, dtype, w, x)
    lim = rounded(dtype, y, b)
    for at in (0, 1280, 2848):
        less = w.copy()
        less[:, at:at + 32] = 0
        assert (np.abs(x @ less.T - y) > lim).mean() > 0.5, at
    swapped = x.copy()
    swapped[:, 64:128] = x[::-1, 64:128]
    assert (np.abs(swapped @ w.T - y) > lim).mean() > 0.5
