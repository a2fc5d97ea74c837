"""Inputs, references and bounds shared by the tests of the chunk operators.

The bounds follow the roundings that the header states, for a product z of K
inputs with A = sum |w||x|:
  activations  fp32: two fp16 terms, 2^-22 each and 2^-50 of the row's largest;
               16-bit: exact but for 2^-39 of the row's largest;
  weights      MXFP4: exact but for 2^-25.  Others: fp32 two terms, 2^-22 and
               2^-36, and as much again for the product of two low terms; fp16
               2^-22 and 2^-25; bf16 one rounding to fp16, 2^-11 and 2^-25;
  sums         every addition in the tensor cores is off by at most 2^-22 of A
               (they truncate, 2^-23, and align a step's products once more):
               K / 16 of them for 16-bit types (twice that with two terms of
               weights), 16 for fp32, whose sums leave every 256 inputs for
               rounded additions (2^-24 each);
  activations' arithmetic: 2^-20 relative (exponential, quotient, erf and the
               products around them, each within 2 ulp).
An output is rounded once, eps / 2 of its type.
"""
import numpy as np
import torch

import oracle
import quantized_weight_streaming_dequant_gb300 as rf
import synthetic as syn
from oracle import chunk as oc

TORCH = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
DTYPES = list(TORCH)
FMTS = [rf.MXFP4, rf.Q4_0, rf.Q8_0, rf.Q4_K]
NAMES = {v: k for k, v in rf.FORMATS.items()}
GATED = (oc.SWIGLU, oc.SWIGLU_CLAMPED)


def randn(rng, shape, dtype, scale=1.0):
    """A device tensor of `dtype` and its exact values."""
    t = torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(TORCH[dtype])
    return t.cuda(), t.double().numpy()


def raw(fmt, n, rows, in_dim, seed, scale_range=None):
    """Stacked raw matrices: the device tensor and (n, rows, in_dim) values."""
    W = syn.quant_matrix(fmt, n * rows, in_dim, seed, scale_range=scale_range)
    return torch.from_numpy(W).cuda(), oc.weights(fmt, W, n, rows, in_dim)


def product_bound(fmt, dtype, in_dim, A, W1, X1, xmax):
    """How far a product may be off; xmax: the rows' largest values, (n, 1)."""
    f32, exact = dtype == "float32", fmt == rf.MXFP4
    rel = {"float32": 2.0 ** -22 + (0 if exact else 2.0 ** -21), "float16": 0 if exact else 2.0 ** -22,
           "bfloat16": 0 if exact else 2.0 ** -11}[dtype]
    steps = 16 if f32 else in_dim / 16 * (2 if dtype == "float16" and not exact else 1)
    rel += (steps + 1) * 2.0 ** -22 + (in_dim / 128 + 32) * 2.0 ** -24
    return A * rel + X1 * 2.0 ** (-36 if f32 and not exact else -25) + W1 * xmax * 2.0 ** (-50 if f32 else -39)


def act_bound(kind, z, bz, u, bu, y, alpha=1.702, limit=7.0):
    """|silu'| <= 1.1, |gelu'| <= 1.13, |d/dz z sigmoid(alpha z)| <= 1.25 (its
    maximum is where silu's is, for every alpha > 0)."""
    own = 2.0 ** -20
    if kind == oc.NONE:
        return bz + own * 2.0 ** -2 * np.abs(y)
    if kind in (oc.SILU, oc.GELU):
        return 1.13 * bz + own * np.abs(z)
    f = np.abs(oc.act(oc.SILU, z)) if kind == oc.SWIGLU else np.abs(np.minimum(z, limit))
    v = np.abs(u) if kind == oc.SWIGLU else np.abs(np.clip(u, -limit, limit)) + 1
    return f * bu + 1.25 * v * bz + 1.25 * bz * bu + own * (f * v + np.abs(y))


def rounded(dtype, y, b):
    """The bound once the value is rounded to its type."""
    return b + torch.finfo(TORCH[dtype]).eps / 2 * (np.abs(y) + b) + 2.0 ** -24 * np.abs(y) + \
        (2.0 ** -25 if dtype == "float16" else 0)


def reference(fmt, dtype, w, x, *, kind=oc.NONE, up=None, bias=None, up_bias=None, residual=None, bx=0.0):
    """(y, bound before rounding) of one matrix; bx: how far x itself may be off."""
    def through(m, b):
        z, A, W1, X1 = oc.product(m, x)
        bound = product_bound(fmt, dtype, m.shape[1], A, W1, X1, np.abs(x).max(1, initial=0)[:, None])
        if not np.isscalar(bx):
            bound = bound + bx @ np.abs(m).T
        if b is not None:
            z = z + b
            bound = bound + 2.0 ** -23 * (np.abs(z) + np.abs(b))
        return z, bound

    z, bz = through(w, bias)
    u, bu = through(up, up_bias) if up is not None else (None, 0.0)
    y = oc.act(kind, z, u)
    b = act_bound(kind, z, bz, u, bu, y)
    if residual is not None:
        y = y + residual
        b = b + 2.0 ** -23 * (np.abs(y) + np.abs(residual))
    return y, b


def moe_reference(fmt, dtype, logits, top_k, gate, up, down, x, *, kind=oc.SWIGLU, gate_bias=None, up_bias=None,
                  down_bias=None, residual=None):
    """(y, bound before rounding) of the routed FFN; weights (n_expert, rows, in)."""
    idx, wt, *_ = oc.route(logits, top_k)
    n_tok, n_embd = x.shape[0], down.shape[1]
    y, b = np.zeros((n_tok, n_embd)), np.zeros((n_tok, n_embd))
    size = np.zeros((n_tok, n_embd))
    pick = lambda t, e: None if t is None else t[e]  # noqa: E731
    for e in np.unique(idx):
        tok, slot = np.nonzero(idx == e)
        h, bh = reference(fmt, dtype, gate[e], x[tok], kind=kind, up=up[e], bias=pick(gate_bias, e), up_bias=pick(up_bias, e))
        # h enters the second product like a row of activations: rounded once to fp16 by 16-bit calls
        if dtype != "float32":
            bh = bh + 2.0 ** -11 * np.abs(h)
        d, bd = reference(fmt, dtype, down[e], h, bias=pick(down_bias, e), bx=bh)
        k = wt[tok, slot][:, None]
        y[tok] += k * d
        b[tok] += k * bd
        size[tok] += np.abs(k * d)
    b += 2.0 ** -20 * size
    if residual is not None:
        y = y + residual
        b += 2.0 ** -23 * (np.abs(y) + np.abs(residual))
    return y, b


def check(got, y, b, dtype, what=""):
    got = got.detach().cpu().double().numpy()
    assert got.shape == y.shape, (what, got.shape, y.shape)
    lim = rounded(dtype, y, b)
    off = np.abs(got - y)
    bad = ~(off <= lim)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}, "
                           f"worst {np.nanmax(off / lim):.3g} of its bound")
    return float(np.max(off / lim)) if off.size else 0.0
