"""Attention over the paged cache in fp64 on the GPU, whole calls at sizes that
the oracle's loops are too slow for (elementary torch operations; no code of
the library)."""
import torch

from oracle import decoder as od


def attention64(cache, table, past, q_start, q, dtype, scale=None, window=0, sinks=None):
    """(out, bound) of rf.attention for the rows of the batch's sequences, whose
    pages are all there.

    The bound is the oracle's, and what it leaves out: weights far below a
    row's largest are held with an absolute error.  A weight w_j times the
    unit 2^ev_j of its values goes to the tensor cores as fp16 numbers in
    which the row's largest is 2^14 (two terms, fp32) or 2^8 (one term) at
    least; fp16's smallest step is 2^-24 and rounds by half of it, so the
    error is up to 2^-39 or 2^-33 of the largest product, for each visible
    position's codes."""
    n_tok, heads, dim = q.shape
    kv = cache.n_kv_heads
    group = heads // kv
    scale = dim ** -0.5 if scale is None else float(scale)
    floor = 2.0 ** -39 if dtype == "float32" else 2.0 ** -33
    new = lambda *s: torch.zeros(s, dtype=torch.float64, device=q.device)  # noqa: E731
    out, mag, xmag, low = new(*q.shape), new(*q.shape), new(n_tok, heads), new(*q.shape)
    for s in range(len(past)):
        a, b, p = int(q_start[s]), int(q_start[s + 1]), int(past[s])
        length = p + b - a
        if b == a:
            continue
        pages = torch.as_tensor(table[s][:-(-length // cache.page_size)], device=q.device).long()
        row = p + torch.arange(b - a, device=q.device)[:, None]
        col = torch.arange(length, device=q.device)[None, :]
        hidden = col > row
        if window:
            hidden |= col <= row - window
        for h in range(heads):
            side = []
            for codes, units in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
                c = codes[pages, h // group].double().flatten(0, 1)[:length]
                u = torch.exp2(units[pages, h // group].double() - 127).flatten().repeat_interleave(32)[:length]
                side += [c, u]
            kc, ku, vc, vu = side
            k, v, x = kc * ku[:, None], vc * vu[:, None], q[a:b, h].double()
            z = (scale * (x @ k.T)).masked_fill_(hidden, -torch.inf)
            top = z.amax(1, keepdim=True)
            w = torch.exp(z - top)
            total = w.sum(1, keepdim=True)
            if sinks is not None:
                total = total + torch.exp(float(sinks[h]) - top)
            out[a:b, h] = w @ v / total
            mag[a:b, h] = w @ v.abs() / total
            xmag[a:b, h] = (abs(scale) * (x.abs() @ k.abs().T)).masked_fill_(hidden, 0).amax(1)
            low[a:b, h] = floor * (w * vu).amax(1, keepdim=True) * ((~hidden).double() @ vc.abs()) / total
    n_pos = max(int(p) + int(q_start[s + 1] - q_start[s]) for s, p in enumerate(past))
    return out, od.attention_bound(dtype, dim, n_pos, out, mag, xmag) + low
