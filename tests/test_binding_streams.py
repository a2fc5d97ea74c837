"""Where the binding's own tensors come from when a call names a stream: from
that stream's memory (CPU: torch's streams and the library are stood in for)."""
import contextlib
import itertools

import pytest
import torch

import quantized_weight_streaming_dequant_gb300 as rf
from quantized_weight_streaming_dequant_gb300.layer import DecoderLayer

SIDE, MAIN = 0x5EED, 0


class Dev(torch.Tensor):
    """A CPU tensor that says it is on the device."""
    is_cuda = True
    used_on = ()

    def record_stream(self, s):
        self.used_on = (*self.used_on, s.cuda_stream)


def dev(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Dev)


class Library:
    """Every call succeeds; sizes are 256 bytes."""

    def __getattr__(self, name):
        return lambda *a: 256 if name.endswith("_bytes") else 0


@pytest.fixture
def made(monkeypatch):
    """[(stream that was current, tensor)] of the binding's allocations."""
    log, current = [], [MAIN]

    class Stream:
        device = None

        def __init__(self, handle=SIDE, *a, **k):
            self.cuda_stream = handle

    @contextlib.contextmanager
    def enter(s):
        current.append(s.cuda_stream)
        yield
        current.pop()

    def new(make):
        def f(*a, **k):
            t = make(*a, **{**k, "device": "cpu"}).as_subclass(Dev)
            log.append((current[-1], t))
            return t
        return f

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream(current[-1]))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: Stream(MAIN))
    monkeypatch.setattr(rf, "_raw_stream", lambda d: current[-1])
    monkeypatch.setattr(rf, "_current_device", lambda: 0)
    monkeypatch.setattr(torch, "empty", new(torch.empty))
    monkeypatch.setattr(torch, "empty_like", new(torch.empty_like))
    monkeypatch.setattr(rf, "lib", lambda: Library())
    keep = {n: getattr(rf, n) for n in ("_DTYPES", "_empty", "_empty_like", "_F32_TYPE") if hasattr(rf, n)}
    rf._look_up()
    log.clear()
    yield log
    for n, v in keep.items():
        setattr(rf, n, v)


class Arena:
    handle = 1
    stream_linear = rf.Arena.stream_linear


def calls():
    W, x, X, lg = dev(4096, dtype=torch.uint8), dev(256), dev(2, 256), dev(8)
    host = torch.zeros(4096, dtype=torch.uint8)
    codes, units = dev(4, 2, 64, 64, dtype=torch.int8), dev(4, 2, 2, dtype=torch.uint8)
    cache = rf.KVCache(codes, codes, units, units)
    i32 = lambda *s: dev(*s, dtype=torch.int32)  # noqa: E731
    batch = rf.KVBatch(i32(1, 4), i32(1), i32(2), 2)
    k, q = dev(2, 2, 64), dev(2, 4, 64)
    f, moe = rf.Q8_0, (rf.Q8_0, lg, 2, W, W, W)
    return {
        "norm": (lambda s: rf.norm_residual(X, X, stream=s), 2),
        "norm of strided rows": (lambda s: rf.norm_residual(dev(2, 300)[:, :256], stream=s), 2),
        "append": (lambda s: rf.kv_append(cache, batch, k, k, q=q, stream=s), 1),
        "read": (lambda s: rf.kv_read(cache, batch, stream=s), 2),
        "attention": (lambda s: rf.attention(cache, batch, q, stream=s), 2),
        "dequantize": (lambda s: rf.dequantize(f, W, 8, stream=s), 1),
        "gemv": (lambda s: rf.gemv(f, W, 0, 4, 256, x, stream=s), 1),
        "gemv_multi": (lambda s: rf.gemv_multi(f, W, 0, 4, 256, X, stream=s), 1),
        "gemm": (lambda s: rf.gemm(f, W, 0, 4, 256, X, stream=s), 2),
        "swiglu": (lambda s: rf.swiglu(x, x, stream=s), 1),
        "gelu": (lambda s: rf.gelu(x, stream=s), 1),
        "gemv_host": (lambda s: rf.gemv_host(f, host, 0, 4, 256, x, stream=s), 1),
        "ffn_swiglu": (lambda s: rf.ffn_swiglu(f, W, W, W, 32, 256, x, stream=s), 2),
        "stream_linear": (lambda s: Arena().stream_linear(f, host, 256, 0, 4, 1, 1, x, stream=s), 1),
        "moe_route": (lambda s: rf.moe_route(lg, 2, stream=s), 2),
        "moe_ffn": (lambda s: rf.moe_ffn(*moe, 32, 256, 1, x, stream=s), 2),
        "moe_ffn_biased": (lambda s: rf.moe_ffn_biased(*moe, None, None, None, 1.0, 1.0, 32, 256, 1, x, stream=s), 2),
        "moe_ffn_host": (lambda s: rf.moe_ffn_host(rf.Q8_0, lg, 2, host, host, host, 32, 256, 1, x, stream=s), 2),
        "moe_ffn_streamed": (lambda s: rf.moe_ffn_streamed(rf.Q8_0, lg, 2, host, host, host, 32, 256, 1, 1, Arena(), x,
                                                           stream=s), 2),
    }


NAMES = ["norm", "norm of strided rows", "append", "read", "attention", "dequantize", "gemv", "gemv_multi", "gemm", "swiglu",
         "gelu", "gemv_host", "ffn_swiglu", "stream_linear", "moe_route", "moe_ffn", "moe_ffn_biased", "moe_ffn_host",
         "moe_ffn_streamed"]
# what a call makes for its kernels alone
PRIVATE = {"attention": 1, "gemm": 1}


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("as_handle", [False, True])
def test_a_call_on_a_stream_takes_that_streams_memory(made, name, as_handle):
    side = SIDE if as_handle else torch.cuda.Stream()
    call, n = calls()[name]
    made.clear()
    call(side)
    assert len(made) == n and all(at == SIDE for at, _ in made)
    # ... and what the caller gets may be used on the current stream, and dropped from there
    assert sum(t.used_on == (MAIN,) for _, t in made) == n - PRIVATE.get(name, 0)


@pytest.mark.parametrize("name", NAMES)
def test_a_call_on_the_current_stream_takes_its_memory(made, name):
    call, n = calls()[name]
    made.clear()
    call(None)
    call(MAIN)
    assert len(made) == 2 * n and all(at == MAIN and t.used_on == () for at, t in made)


@pytest.mark.parametrize("fmt,n_tok", [*itertools.product([rf.Q8_0, rf.Q6_K], [1, 5, 20])])
def test_a_decoder_layer_on_a_stream_takes_that_streams_memory(made, fmt, n_tok):
    W, norm = dev(4096, dtype=torch.uint8), dev(256)
    codes, units = dev(4, 2, 64, 64, dtype=torch.int8), dev(4, 2, 2, dtype=torch.uint8)
    cache = rf.KVCache(codes, codes, units, units)
    i32 = lambda *s: dev(*s, dtype=torch.int32)  # noqa: E731
    batch = rf.KVBatch(i32(1, 4), i32(1), i32(2), n_tok)
    layer = DecoderLayer(fmt, 256, 512, 4, 2, 64, W, W, W, W, W, W, W, norm, norm)
    made.clear()
    o = layer.step(dev(n_tok, 256), dev(n_tok, 256), cache, batch, stream=torch.cuda.Stream())
    layer.finish(o["residual"], o["delta"], stream=torch.cuda.Stream())
    assert len(made) > 10 and all(at == SIDE for at, _ in made)
