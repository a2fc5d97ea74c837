"""The decoder layer's attention, FFN and calls against fp64: attention over the
oracle's cache, the SwiGLU hidden vector, ragged batches, and a captured decode
loop."""
import numpy as np
import pytest
import torch

import oracle
import quantized_weight_streaming_dequant_gb300 as rf
from attention64 import attention64
from decoder_helpers import i32
from gpu_helpers import derived_gemm_bound, dev_tensor, gemv_tol, swiglu_h_tol
from oracle import decoder as od
from test_gpu_decoder_layer import D, FF, HD, NH, NK, PAGE, make, project_check

pytestmark = pytest.mark.gpu

FORMATS = [rf.Q8_0, rf.Q4_0, rf.MXFP4, rf.Q4_K, rf.Q6_K]


class Checked:
    """A layer, its cache and the oracle's."""

    def __init__(self, fmt, rng, table, **kw):
        self.fmt, self.table = fmt, np.asarray(table, np.int32)
        self.layer, self.W, self.norms, self.tab = make(fmt, rng, **kw)
        self.cache = rf.KVCache.empty(int(self.table.max()) + 1, NK, PAGE, HD)
        self.ref = od.Cache(*(t.cpu().numpy() for t in (self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale)))

    def rotated(self, x, past, q_start):
        out = np.array(x, np.float32)
        for s, p in enumerate(past):
            for t in range(q_start[s], q_start[s + 1]):
                at = p + t - q_start[s]
                out[t] = od.rotate(x[t], self.tab["cos"][at], self.tab["sin"][at], False)
        return out

    def project(self, name, rows, cols, x):
        """The fp64 projections of x and their bound, as the layer makes them."""
        W = self.W[name]
        y = np.stack([oracle.gemv(self.fmt, W, 0, rows, cols, r) for r in x])
        if len(x) > 8 and self.fmt != rf.Q6_K:
            return y, derived_gemm_bound(self.fmt, W, 0, rows, cols, x)
        return y, np.stack([gemv_tol(self.fmt, W, 0, rows, cols, r) for r in x])

    def check(self, o, past, new):
        """Every stage of a step on that stage's own inputs."""
        q_start = np.concatenate([[0], np.cumsum(new)]).astype(int)
        got = {k: v.double().cpu().numpy() for k, v in o.items()}
        x32 = o["x"].cpu().numpy()
        for name, rows, key in (("wq", NH * HD, "q"), ("wk", NK * HD, "k"), ("wv", NK * HD, "v")):
            project_check(self.fmt, self.W[name], rows, D, x32, got[key])
        q = self.rotated(o["q"].cpu().numpy(), past, q_start)
        assert np.array_equal(o["q_rot"].cpu().numpy(), q)
        self.ref.append(self.table, past, q_start, self.rotated(o["k"].cpu().numpy(), past, q_start), o["v"].cpu().numpy())
        for got_c, want in zip((self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale), self.ref.codes + self.ref.scales):
            assert np.array_equal(got_c.cpu().numpy(), want)
        ref, bound = attention64(self.cache, self.table, past, q_start, o["q_rot"], "float32", window=self.layer.window,
                                 sinks=self.layer.sinks)
        assert ((o["attn"].double() - ref).abs() <= bound).all()
        project_check(self.fmt, self.W["wo"], D, NH * HD, o["attn"].cpu().numpy(), got["o"])
        y32 = o["y"].cpu().numpy()
        g, tg = self.project("w_gate", FF, D, y32)
        u, tu = self.project("w_up", FF, D, y32)
        assert (np.abs(got["h"].reshape(g.shape) - g / (1 + np.exp(-g)) * u) <= swiglu_h_tol(g, u, tg, tu)).all()
        project_check(self.fmt, self.W["w_down"], D, FF, o["h"].cpu().numpy(), got["delta"])


def residual(rng, n):
    return dev_tensor(rng.standard_normal((n, D)).astype(np.float32))


@pytest.mark.parametrize("fmt", FORMATS)
def test_prompt_and_tokens(fmt):
    rng = np.random.default_rng([fmt, 1])
    c = Checked(fmt, rng, [[5, 2, 7, 0]], window=48 if fmt == rf.Q4_0 else 0)
    past = 0
    for n in (130, 1, 5, 1, 20):                                # the GEMM, the GEMV and its batched form
        batch = rf.KVBatch(i32(c.table), i32([past]), i32([0, n]), n)
        o = c.layer.step(residual(rng, n), residual(rng, n), c.cache, batch, prev_post=c.layer.post_ffn, max_len=past + n)
        c.check(o, [past], [n])
        past += n
    assert rf.device_status() == rf.OK


@pytest.mark.parametrize("window", [0, 300])
def test_a_prompt_through_the_tiles(window):
    rng = np.random.default_rng([31, window])
    c = Checked(rf.Q8_0, rng, [[4, 0, 7, 2, 6, 1, 5, 3]], window=window)
    past = 0
    for n in (500, 1, 9):
        batch = rf.KVBatch(i32(c.table), i32([past]), i32([0, n]), n)
        o = c.layer.step(residual(rng, n), residual(rng, n), c.cache, batch, max_len=past + n)
        plan = rf.debug_attention_plan(c.cache, batch, o["q_rot"], window=window, max_len=past + n)
        assert plan["tiles"] == (n == 500)
        c.check(o, [past], [n])
        past += n
    assert rf.device_status() == rf.OK


@pytest.mark.parametrize("fmt", [rf.Q8_0, rf.MXFP4])
@pytest.mark.parametrize("steps", [[[1, 1, 1]], [[40, 3, 70], [1, 1, 1]], [[5, 0, 2], [0, 6, 1], [1, 1, 1], [9, 1, 30]]])
def test_ragged_batches(fmt, steps):
    rng = np.random.default_rng([fmt, len(steps)])
    c = Checked(fmt, rng, [[3, 8, 1], [0, 5, 4], [7, 2, 6]])
    past = [0, 0, 0]
    for new in steps:
        q_start = np.concatenate([[0], np.cumsum(new)])
        batch = rf.KVBatch(i32(c.table), i32(past), i32(q_start), int(q_start[-1]))
        o = c.layer.step(residual(rng, sum(new)), None, c.cache, batch)
        c.check(o, past, new)
        past = [p + n for p, n in zip(past, new)]
    assert rf.device_status() == rf.OK


@pytest.mark.parametrize("n_seq", [1, 3])
def test_a_captured_layer_decodes(n_seq):
    """One capture of a step serves the next tokens: lengths are read on the device."""
    rng = np.random.default_rng([30, n_seq])
    c = Checked(rf.Q8_0, rng, np.arange(3 * n_seq).reshape(n_seq, 3)[:, ::-1])
    past, starts = i32([0] * n_seq), np.arange(n_seq + 1)
    batch = rf.KVBatch(i32(c.table), past, i32(starts), n_seq)
    res, delta = residual(rng, n_seq), residual(rng, n_seq)

    def step():
        o = c.layer.step(res, delta, c.cache, batch, prev_post=c.layer.post_ffn)
        past.add_(1)
        return o

    step()                                                      # first use outside a capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step()
    for t in (c.cache.k, c.cache.v, c.cache.k_scale, c.cache.v_scale, past):
        t.zero_()
    for i in range(40):                                         # past the first block of 32
        res.copy_(residual(rng, n_seq))
        delta.copy_(residual(rng, n_seq))
        graph.replay()
        torch.cuda.synchronize()
        c.check(o, [i] * n_seq, [1] * n_seq)
    assert rf.device_status() == rf.OK
