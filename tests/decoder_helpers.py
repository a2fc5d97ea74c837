"""Inputs and checks shared by the decoder-operator tests."""
import numpy as np
import torch

import quantized_weight_streaming_dequant_gb300 as rf
from oracle import decoder as od

TORCH = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
DTYPES = list(TORCH)


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def randn(rng, shape, dtype="float32", scale=1.0):
    """A device tensor of `dtype` and its exact values in fp64."""
    t = torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(TORCH[dtype])
    return t.cuda(), t.double().numpy()


def strided(t, pad_tok=0, pad_head=0):
    """The same (tok, head, dim) values in a wider buffer."""
    n, h, d = t.shape
    wide = torch.full((n, h + pad_tok, d + pad_head), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, :h, :d] = t
    return wide[:, :h, :d]


class Setup:
    """A cache, its page table and a ragged batch, on both sides."""

    def __init__(self, rng, past, new, kv, dim, page, codes=True, pad_tokens=0, spare=2, width=0, scales=(118, 123)):
        self.past, self.new = list(past), list(new)
        n_seq = len(past)
        need = [max(1, -(-(p + n) // page)) for p, n in zip(past, new)]
        width = max(width, max(need))
        n_pages = sum(need) + spare
        order = rng.permutation(n_pages)
        self.table = np.full((n_seq, width), -1, np.int32)      # entries past a sequence name no page
        at = 0
        for s, m in enumerate(need):
            self.table[s, :m] = order[at:at + m]
            at += m
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.n_tok = int(self.q_start[-1]) + pad_tokens
        shape, sc = (n_pages, kv, page, dim), (n_pages, kv, page // 32)
        k = np.clip(np.rint(30 * rng.standard_normal(shape)), -127, 127).astype(np.int8) if codes else np.zeros(shape, np.int8)
        v = np.clip(np.rint(30 * rng.standard_normal(shape)), -127, 127).astype(np.int8) if codes else np.zeros(shape, np.int8)
        ks = rng.integers(*scales, sc).astype(np.uint8)
        vs = rng.integers(*scales, sc).astype(np.uint8)
        # blocks that no sequence has reached hold NaN units
        used = np.zeros(sc[:1] + sc[2:], bool)
        for s, m in enumerate(need):
            for b in range(-(-(past[s] + new[s]) // 32)):
                used[self.table[s, b * 32 // page], b % (page // 32)] = True
        ks[~np.broadcast_to(used[:, None], sc)] = 255
        vs[~np.broadcast_to(used[:, None], sc)] = 255
        self.ref = od.Cache(k, v, ks, vs)
        self.upload()

    def upload(self):
        t = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        self.cache = rf.KVCache(t(self.ref.codes[0]), t(self.ref.codes[1]), t(self.ref.scales[0]), t(self.ref.scales[1]))
        self.batch = rf.KVBatch(i32(self.table), i32(self.past), i32(self.q_start), self.n_tok)

    def same_cache(self):
        got = (self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale)
        for g, w, what in zip(got, self.ref.codes + self.ref.scales, ("k", "v", "k_scale", "v_scale")):
            g = g.cpu().numpy()
            # codes of a block that is marked are not defined
            if what in ("k", "v"):
                nan = np.repeat(self.ref.scales["kv".index(what)] == 255, 32, axis=2)[..., None]
                g, w = np.where(nan, 0, g), np.where(nan, 0, w)
            assert np.array_equal(g, w), f"{what} differs in {np.argwhere(g != w)[:4].tolist()}"


def check_attention(su, q, q64, dtype, scale=None, window=0, sinks=None, max_len=0, **kw):
    """rf.attention against the oracle within the derived bound; returns it."""
    dim = q.shape[2]
    out = rf.attention(su.cache, su.batch, q, scale=scale, window=window, max_len=max_len,
                       sinks=None if sinks is None else torch.from_numpy(np.asarray(sinks, np.float32)).cuda(), **kw)
    ref, mag, xmag = od.attention(su.ref, su.table, su.past, su.q_start, su.n_tok, q64,
                                  dim ** -0.5 if scale is None else np.float32(scale), window, sinks)
    n_pos = max(p + n for p, n in zip(su.past, su.new))
    bound = od.attention_bound(dtype, dim, n_pos, ref, mag, xmag)
    got = out.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    err = np.abs(got - ref)
    worst = np.nanmax(err / bound) if err.size else 0.0
    assert worst <= 1.0, (worst, np.argwhere(err > bound)[:5].tolist())
    return out


def by_tiles(su, heads, window=0, max_len=0):
    """Whether the call goes through the 128-row tiles: 96 rows (tokens x heads
    of a group) a sequence and half a million row-position pairs."""
    per = -(-su.n_tok // len(su.past))
    rows = per * heads // su.ref.heads
    seen = max_len or su.table.shape[1] * su.ref.page
    return rows >= 96 and rows * min(seen, window + per if window else seen) * len(su.past) >= 5e5
