"""CPU oracle of what a decoder layer computes around its projections -- TEST
INFRASTRUCTURE, numpy in fp64, sharing no code with the CUDA path.

The cache's codes are defined by fp32 roundings (the rotation's products and
sums, then ties to even), so ``append`` follows them in fp32 numpy, where each
operation rounds once; norms and attention are in fp64.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
E_MIN, E_MAX, E_NAN = 87, 167, 255


def norm_residual(x, residual, post_weight, gate, scale, weight, eps):
    """(r, y): t = x or its norm, r = residual + scale * gate * t, y = norm of r."""
    def rms(a, w):
        a = a / np.sqrt(np.mean(a * a, axis=-1, keepdims=True) + eps)
        return a if w is None else a * np.asarray(w, np.float64)

    r = 0.0 if residual is None else np.asarray(residual, np.float64)
    if x is not None:
        t = np.asarray(x, np.float64)
        if post_weight is not None:
            t = rms(t, post_weight)
        if gate is not None:
            t = t * np.asarray(gate, np.float64)
        r = r + float(scale) * t
    return r, rms(r, weight)


def rotate(x, cos, sin, pairs):
    """x (heads, dim) fp32 by one position's tables (rot / 2,): fp32, each
    product and sum rounded on its own."""
    x = np.array(x, np.float32)
    half = 0 if cos is None else len(cos)
    if half == 0:
        return x
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
    xa, xb = x[:, a].copy(), x[:, b].copy()
    c, s = np.asarray(cos, np.float32), np.asarray(sin, np.float32)
    x[:, a] = xa * c - xb * s
    x[:, b] = xb * c + xa * s
    return x


def unit(E):
    """2^(E-127); NaN for 255."""
    E = np.asarray(E, np.int64)
    return np.where(E == E_NAN, np.nan, np.ldexp(1.0, E - 127))


def scale_byte(amax: float) -> int:
    if not np.isfinite(amax):
        return E_NAN
    for E in range(E_MIN, E_MAX + 1):
        if amax <= 127.0 * 2.0 ** (E - 127):
            return E
    return E_NAN


class Cache:
    """The cache as numpy arrays, one token at a time."""

    def __init__(self, k, v, k_scale, v_scale):
        self.codes = [np.array(k), np.array(v)]
        self.scales = [np.array(k_scale), np.array(v_scale)]
        self.n_pages, self.heads, self.page, self.dim = self.codes[0].shape

    def at(self, table_row, pos):
        """(page, offset) of a position, or None."""
        i = pos // self.page
        if pos < 0 or i >= len(table_row) or not 0 <= table_row[i] < self.n_pages:
            return None
        return int(table_row[i]), pos % self.page

    def append(self, table, past, q_start, k, v):
        """k (already rotated) and v, fp32 (n_tok, heads, dim)."""
        for s in range(len(past)):
            n, t0 = int(q_start[s + 1] - q_start[s]), int(q_start[s])
            j = 0
            while j < n:
                pos = int(past[s]) + j
                m = min(n - j, BLOCK - pos % BLOCK)      # the call's tokens in this block
                where = self.at(table[s], pos)
                if where is not None:
                    page, off = where
                    held = off % BLOCK
                    for side, x in enumerate((k, v)):
                        for h in range(self.heads):
                            self._block(side, page, h, off, held, x[t0 + j:t0 + j + m, h])
                j += m

    def _block(self, side, page, h, off, held, x):
        x = np.asarray(x, np.float64)
        codes, scales, sub = self.codes[side], self.scales[side], off // BLOCK
        E = scale_byte(float(np.abs(x).max()) if not np.isnan(x).any() else np.nan)
        old = int(scales[page, h, sub])
        if held:
            E = max(E, old)
        if E != E_NAN:
            if held and E > old:
                was = codes[page, h, off - held:off].astype(np.float64)
                codes[page, h, off - held:off] = np.rint(was * 2.0 ** (old - E)).astype(np.int8)
            codes[page, h, off:off + len(x)] = np.rint(x * 2.0 ** (127 - E)).astype(np.int8)
        scales[page, h, sub] = E

    def values(self, table_row, pos, side):
        """(heads, dim) fp64 values at a position, or None."""
        where = self.at(table_row, pos)
        if where is None:
            return None
        page, off = where
        return self.codes[side][page, :, off].astype(np.float64) * unit(self.scales[side][page, :, off // BLOCK])[:, None]


def attention(cache, table, past, q_start, n_tok, q, scale, window=0, sinks=None):
    """(out, mag, xmag): the output (n_tok, heads, dim), sum w|v| / sum w, and
    per (token, head) the largest scale * sum |q||k| over the visible
    positions: what the error bounds need."""
    q = np.asarray(q, np.float64)
    heads, dim = q.shape[1], q.shape[2]
    group = heads // cache.heads
    out, mag, xmag = np.zeros(q.shape), np.zeros(q.shape), np.zeros((n_tok, heads))
    for s in range(len(past)):
        n = int(past[s]) + int(q_start[s + 1]) - int(q_start[s])
        there = np.array([cache.at(table[s], j) is not None for j in range(max(n, 0))], bool)
        zero = np.zeros((cache.heads, dim))
        keys, vals = (np.stack([cache.values(table[s], j, side) if there[j] else zero for j in range(n)])
                      if n > 0 else None for side in (0, 1))
        for t in range(int(q_start[s]), int(q_start[s + 1])):
            last = int(past[s]) + t - int(q_start[s])
            pos = np.arange(max(0, last - window + 1) if window else 0, last + 1)
            pos = pos[there[pos]]
            if not len(pos):
                continue
            k, v = keys[pos], vals[pos]                                    # (n, kv heads, dim)
            for h in range(heads):
                kh, vh = k[:, h // group], v[:, h // group]
                z = float(scale) * (kh @ q[t, h])
                top = z.max()
                w = np.exp(z - top)
                total = w.sum()
                if sinks is not None:
                    total = total + np.exp(min(float(sinks[h]) - top, 700.0))
                out[t, h] = w @ vh / total
                mag[t, h] = w @ np.abs(vh) / total
                xmag[t, h] = abs(float(scale)) * (np.abs(kh) @ np.abs(q[t, h])).max()
    return out, mag, xmag


def attention_bound(dtype, dim, n_pos, out, mag, xmag):
    """Error bound of the attention kernels' arithmetic per output element.

    Score error in log2 units: q enters as two fp16 terms (2^-21 relative to
    the row's maximum, so to sum|q||k| with a factor of dim / sqrt(dim) at
    most, taken as 2^-19) or exactly; each of up to 2 * dim / 16 tensor sums
    truncates (2^-23); the scale, the exponent's argument and the unit each
    round (2^-22 of up to |x| + 64).  A weight's relative error is ln 2 times
    that, plus 2^-21 for the exponential and the two-term split, or 2^-11 for
    the one fp16 rounding of 16-bit types.  Numerator and denominator each
    carry it; sums over blocks round once per block of 32 positions and once
    per join (2^-23 each, taken over n_pos / 8 + 64).  The output rounds once.
    """
    x = 1.4427 * xmag[..., None]
    ex = x * (2.0 ** -19 + dim / 8 * 2.0 ** -23) + 2.0 ** -22 * (x + 64.0)
    ew = 0.6932 * ex + 2.0 ** -21 + (n_pos / 8 + 64) * 2.0 ** -23
    bound = 2.0 * ew * mag
    if dtype != "float32":
        bound = bound + 2.0 ** -11 * mag + (2.0 ** -8 if dtype == "bfloat16" else 2.0 ** -10) * abs(out) + 2.0 ** -24
    return bound + 1e-30
