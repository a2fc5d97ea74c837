"""Compositions of the C ABI calls into the decode steps the library serves.

Nothing here computes: each function only sequences C ABI launches (through
the binding) on one stream.

DenseLayer -- one dense decode layer held resident in HBM: the Q, K and V
  projections of x in one batched launch, the O projection of the attention
  output, then the two-phase SwiGLU FFN (gate/up with the SwiGLU epilogue, then
  down).  The output of the attention between QKV and O is an input here.
DecoderLayer -- the whole decoder layer over a paged KV cache, from residual
  stream to residual stream, for single tokens and chunks of a prompt: norm,
  Q/K/V, rotation and append, attention, O, norm, SwiGLU FFN.
StreamedFFN -- a dense FFN whose weights stay in page-locked host memory: up
  (host-streamed), GELU, down (host-streamed), all through one arena; or the
  same FFN read in place over the host link (zero copy).
"""
from __future__ import annotations

from dataclasses import dataclass

import quantized_weight_streaming_dequant_gb300 as rf


@dataclass
class DenseLayer:
    fmt: int
    d_model: int
    d_ff: int
    wq: object
    wk: object
    wv: object
    wo: object
    w_gate: object
    w_up: object
    w_down: object

    def step(self, x, attn, x_ffn, out, stream=None, chain: bool = True):
        """out: dict of device tensors q, k, v, o, h, y (preallocated), and
        optionally hd, an ffn_workspace for h's digits.  With
        `chain`, each launch copies its (static) weights while the previous
        kernel on the stream drains (RF_CHAIN)."""
        d = self.d_model
        fl = rf.CHAIN if chain else 0
        rf.gemv_batch(self.fmt, d, [(self.wq, 0, d, x, out["q"]), (self.wk, 0, d, x, out["k"]),
                                    (self.wv, 0, d, x, out["v"])], stream=stream, flags=fl)
        rf.gemv(self.fmt, self.wo, 0, d, d, attn, out["o"], stream=stream, flags=fl)
        rf.ffn_swiglu(self.fmt, self.w_gate, self.w_up, self.w_down, self.d_ff, d, x_ffn,
                      out["y"], out["h"], stream=stream, flags=fl, workspace=out.get("hd"))

    def weight_bytes(self) -> int:
        rb_d = rf.row_bytes(self.fmt, self.d_model)
        rb_ff = rf.row_bytes(self.fmt, self.d_ff)
        return 4 * self.d_model * rb_d + 2 * self.d_ff * rb_d + self.d_model * rb_ff

    @staticmethod
    def launches_per_step() -> int:
        return 4   # QKV batch, O, gate/up+SwiGLU, down


@dataclass
class DecoderLayer:
    """One decoder layer.  Weights are quantized matrices (rows x inputs): wq
    (n_heads * head_dim, d_model), wk and wv (n_kv_heads * head_dim, d_model),
    wo (d_model, n_heads * head_dim), w_gate and w_up (d_ff, d_model), w_down
    (d_model, d_ff).  Norm weights, sinks and the rotation's tables (n_pos,
    rot / 2) are float32; activations are float32, (n_tok, d_model)."""
    fmt: int
    d_model: int
    d_ff: int
    n_heads: int
    n_kv_heads: int
    head_dim: int
    wq: object
    wk: object
    wv: object
    wo: object
    w_gate: object
    w_up: object
    w_down: object
    norm_attn: object
    norm_ffn: object
    cos: object = None
    sin: object = None
    rope: int = rf.ROPE_HALF
    post_attn: object = None     # norms of the blocks' outputs, or None
    post_ffn: object = None
    sinks: object = None
    window: int = 0
    eps: float = 1e-5
    residual_scale: float = 1.0

    def _project(self, W, rows, in_dim, x, stream):
        """x (n_tok, in_dim) through W: the GEMV for one token, its batched
        form for up to eight (and for every format), the GEMM for chunks."""
        n_tok = x.shape[0]
        if n_tok <= 8:
            return rf.gemv_multi(self.fmt, W, 0, rows, in_dim, x, stream=stream)
        if self.fmt == rf.Q6_K:
            y = rf._new_f32(stream, (n_tok, rows), x)
            for t in range(0, n_tok, 8):
                rf.gemv_multi(self.fmt, W, 0, rows, in_dim, x[t:t + 8], y[t:t + 8], stream=stream)
            return y
        return rf.gemm(self.fmt, W, 0, rows, in_dim, x, stream=stream)

    def step(self, residual, delta, cache, batch, prev_post=None, max_len=0, stream=None):
        """The batch's tokens through the layer.  residual: the stream before
        it; delta: the previous layer's FFN output, not yet added (None for
        the first layer), prev_post its norm weights.  Returns a dict: the
        new residual and delta for the next layer ("residual", "delta"; add
        the last one with `finish`), and the values in between."""
        d, hd, nh, nk = self.d_model, self.head_dim, self.n_heads, self.n_kv_heads
        n_tok = batch.n_tok
        s, alpha = stream, self.residual_scale
        o = {}
        o["in"], o["x"] = rf.norm_residual(residual, delta, post_weight=prev_post, scale=alpha,
                                           weight=self.norm_attn, eps=self.eps, stream=s)
        if n_tok == 1:
            q, k, v = (rf._new_f32(s, n, residual) for n in (nh * hd, nk * hd, nk * hd))
            x = o["x"].view(-1)
            rf.gemv_batch(self.fmt, d, [(self.wq, 0, nh * hd, x, q), (self.wk, 0, nk * hd, x, k),
                                        (self.wv, 0, nk * hd, x, v)], stream=s)
        else:
            q = self._project(self.wq, nh * hd, d, o["x"], s)
            k = self._project(self.wk, nk * hd, d, o["x"], s)
            v = self._project(self.wv, nk * hd, d, o["x"], s)
        o["q"], o["k"], o["v"] = q.view(n_tok, nh, hd), k.view(n_tok, nk, hd), v.view(n_tok, nk, hd)
        o["q_rot"] = rf.kv_append(cache, batch, o["k"], o["v"], q=o["q"], cos=self.cos, sin=self.sin,
                                  rope=self.rope, stream=s, flags=rf.CHAIN if n_tok == 1 else 0)
        o["attn"] = rf.attention(cache, batch, o["q_rot"], window=self.window, sinks=self.sinks,
                                 max_len=max_len, stream=s, flags=rf.CHAIN)
        o["o"] = self._project(self.wo, d, nh * hd, o["attn"].view(n_tok, nh * hd), s)
        o["residual"], o["y"] = rf.norm_residual(o["in"], o["o"], post_weight=self.post_attn,
                                                 scale=alpha, weight=self.norm_ffn, eps=self.eps, stream=s)
        if n_tok == 1:
            y, o["h"] = rf.ffn_swiglu(self.fmt, self.w_gate, self.w_up, self.w_down, self.d_ff, d,
                                      o["y"].view(-1), stream=s)
            o["delta"] = y.view(1, d)
        else:
            g = self._project(self.w_gate, self.d_ff, d, o["y"], s)
            u = self._project(self.w_up, self.d_ff, d, o["y"], s)
            o["h"] = rf.swiglu(g, u, stream=s)
            o["delta"] = self._project(self.w_down, d, self.d_ff, o["h"], s)
        return o

    def finish(self, residual, delta, weight=None, stream=None):
        """After the last layer: its delta added, and the final norm (of
        `weight`): (residual, normed)."""
        return rf.norm_residual(residual, delta, post_weight=self.post_ffn, scale=self.residual_scale,
                                weight=weight, eps=self.eps, stream=stream)


@dataclass
class StreamedFFN:
    fmt: int
    d_model: int
    d_ff: int
    host_up: object     # page-locked [d_ff][d_model] bytes
    host_down: object   # page-locked [d_model][d_ff] bytes

    def step(self, arena, x, u, h, y, block_rows, depth, stream=None):
        arena.stream_linear(self.fmt, self.host_up, self.d_model, 0, self.d_ff, block_rows, depth,
                            x, u, stream=stream)
        rf.gelu(u, h, stream=stream)
        arena.stream_linear(self.fmt, self.host_down, self.d_ff, 0, self.d_model, block_rows,
                            depth, h, y, stream=stream)

    def step_zero_copy(self, x, u, h, y, stream=None):
        """The same FFN with both projections read in place from page-locked
        host memory (rf_gemv_host): no arena, no copy engine."""
        rf.gemv_host(self.fmt, self.host_up, 0, self.d_ff, self.d_model, x, u, stream=stream)
        rf.gelu(u, h, stream=stream)
        rf.gemv_host(self.fmt, self.host_down, 0, self.d_model, self.d_ff, h, y, stream=stream)

    def weight_bytes(self) -> int:
        return (self.d_ff * rf.row_bytes(self.fmt, self.d_model) +
                self.d_model * rf.row_bytes(self.fmt, self.d_ff))
