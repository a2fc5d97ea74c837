"""CPU oracle of the operators of a chunk of tokens -- TEST INFRASTRUCTURE,
numpy in fp64 over the C oracle's dequantized weights, sharing no code with the
CUDA path.

Besides each result it gives what a bound on its rounding needs: for a product
sum_i w_i x_i the sums of |w_i| |x_i|, |w_i| and |x_i|.
"""
from __future__ import annotations

import numpy as np

import oracle

NONE, SILU, GELU, SWIGLU, SWIGLU_CLAMPED = range(5)


def weights(fmt: int, W, n: int, rows: int, in_dim: int) -> np.ndarray:
    """(n, rows, in_dim) values of stacked raw matrices."""
    return np.asarray(oracle.dequantize(fmt, W), np.float64).reshape(n, rows, in_dim)


def route(logits, top_k: int):
    """(idx, w, offsets, order, place) of (n_tok, n_expert) logits."""
    x = np.asarray(logits, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    n_tok, n_expert = x.shape
    idx = np.array([sorted(range(n_expert), key=lambda e: (-row[e], e))[:top_k] for row in x], np.int32)
    idx = idx.reshape(n_tok, top_k)
    with np.errstate(invalid="ignore"):
        e = np.exp(np.take_along_axis(x, idx, 1) - np.take_along_axis(x, idx[:, :1], 1))
        w = e / e.sum(1, keepdims=True)
    flat = idx.ravel()
    order = np.array(sorted(range(flat.size), key=lambda f: (flat[f], f)), np.int32)
    place = np.empty_like(order)
    place[order] = np.arange(flat.size)
    offsets = np.array([np.sum(flat < e) for e in range(n_expert + 1)], np.int32)
    return idx, w, offsets, order, place


def product(w, x):
    """z = w x for w (rows, in), x (n, in): (z, sum |w||x|, sum |w|, sum |x|)."""
    x = np.asarray(x, np.float64)
    return x @ w.T, np.abs(x) @ np.abs(w).T, np.abs(w).sum(1)[None], np.abs(x).sum(1)[:, None]


def act(kind: int, z, u=None, alpha: float = 1.702, limit: float = 7.0):
    def sigmoid(t):
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-t))

    if kind == SILU:
        return z * sigmoid(z)
    if kind == GELU:
        from scipy.special import erfc
        return 0.5 * z * erfc(-z / np.sqrt(2.0))
    if kind == SWIGLU:
        return z * sigmoid(z) * u
    if kind == SWIGLU_CLAMPED:
        z, u = np.minimum(z, limit), np.clip(u, -limit, limit)
        return z * sigmoid(alpha * z) * (u + 1.0)
    return z
