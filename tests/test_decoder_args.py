"""Argument checks of the operators between the projections: made on the host
before anything is enqueued, so they need no GPU (the pointers are never read)."""
import ctypes

import pytest

import quantized_weight_streaming_dequant_gb300 as rf

OK, INVALID, UNSUPPORTED, CUDA, MISALIGNED, TOO_LARGE = 0, 1, 2, 5, 8, 9
P = 1 << 20   # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def L():
    from quantized_weight_streaming_dequant_gb300 import build
    build.build()
    return rf.lib()


def norm(L, **kw):
    a = dict(dtype=rf.F32, n_tok=0, n=64, x=P, ldx=64, post=None, gate=None, ldg=0, scale=1.0, res=P, ldr=64, ro=P,
             ldro=64, w=None, y=P, ldy=64, eps=1e-5, flags=0)
    a.update(kw)
    return L.rf_norm_residual(a["dtype"], a["n_tok"], a["n"], a["x"], a["ldx"], a["post"], a["gate"], a["ldg"],
                              a["scale"], a["res"], a["ldr"], a["ro"], a["ldro"], a["w"], a["y"], a["ldy"], a["eps"],
                              a["flags"], None)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(dtype=7), UNSUPPORTED), (dict(n=0), INVALID), (dict(n_tok=-1), INVALID),
    (dict(n_tok=1, x=None, res=None), INVALID), (dict(n_tok=1, ro=None, y=None), INVALID), (dict(ldx=63), INVALID),
    (dict(ldr=63), INVALID), (dict(ldro=63), INVALID), (dict(ldy=63), INVALID), (dict(gate=P, ldg=63), INVALID),
    (dict(gate=P, ldg=64), OK), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(flags=2), INVALID), (dict(x=P + 2), MISALIGNED),
    (dict(x=P + 2, dtype=rf.BF16), OK), (dict(y=P + 1, dtype=rf.F16), MISALIGNED), (dict(w=P + 2), MISALIGNED),
    (dict(n=32769, ldx=40000, ldr=40000, ldro=40000, ldy=40000), TOO_LARGE), (dict(n_tok=2 ** 31), TOO_LARGE)])
def test_norm_arguments(L, kw, want):
    assert norm(L, **kw) == want


def cache(**kw):
    a = dict(k=P, v=P, ks=P, vs=P, n_pages=10, page=64, kv=2, dim=64, reserved=0)
    a.update(kw)
    return rf.KVCacheStruct(a["k"], a["v"], a["ks"], a["vs"], a["n_pages"], a["page"], a["kv"], a["dim"], a["reserved"])


def batch(**kw):
    a = dict(table=P, past=P, q_start=P, stride=4, width=4, n_seq=1, n_tok=0, reserved=0)
    a.update(kw)
    return rf.KVBatchStruct(a["table"], a["past"], a["q_start"], a["stride"], a["width"], a["n_seq"], a["n_tok"],
                            a["reserved"])


def ref(s):
    return ctypes.byref(s) if s is not None else None


def append(L, c, b, **kw):
    a = dict(dtype=rf.F32, k=P, klt=128, klh=64, v=P, vlt=128, vlh=64, q=P, qlt=256, qlh=64, qo=P, olt=256, olh=64,
             heads=4, cos=P, sin=P, n_pos=100, rot=64, style=rf.ROPE_HALF, flags=0)
    a.update(kw)
    return L.rf_kv_append(ref(c), ref(b), a["dtype"], a["k"], a["klt"], a["klh"], a["v"], a["vlt"], a["vlh"], a["q"],
                          a["qlt"], a["qlh"], a["qo"], a["olt"], a["olh"], a["heads"], a["cos"], a["sin"], a["n_pos"],
                          a["rot"], a["style"], a["flags"], None)


def attend(L, c, b, **kw):
    a = dict(dtype=rf.F32, q=P, qlt=256, qlh=64, heads=4, scale=0.1, window=0, sinks=None, out=P, olt=256, olh=64,
             max_len=0, ws=None, ws_bytes=0, flags=0)
    a.update(kw)
    return L.rf_attention(ref(c), ref(b), a["dtype"], a["q"], a["qlt"], a["qlh"], a["heads"], a["scale"], a["window"],
                          a["sinks"], a["out"], a["olt"], a["olh"], a["max_len"], a["ws"], a["ws_bytes"], a["flags"],
                          None)


BAD_CACHE = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(ks=None), INVALID), (dict(vs=None), INVALID),
             (dict(n_pages=0), INVALID), (dict(n_pages=2 ** 31), INVALID), (dict(page=16), INVALID),
             (dict(page=96), INVALID), (dict(page=512), INVALID), (dict(kv=0), INVALID), (dict(kv=1025), INVALID),
             (dict(dim=0), INVALID), (dict(dim=72), INVALID), (dict(dim=272), INVALID), (dict(reserved=1), INVALID),
             (dict(k=P + 8), MISALIGNED), (dict(v=P + 4), MISALIGNED),
             (dict(n_pages=2 ** 31 - 1, kv=1024), TOO_LARGE)]
BAD_BATCH = [(dict(table=None), INVALID), (dict(past=None), INVALID), (dict(q_start=None), INVALID),
             (dict(n_seq=0), INVALID), (dict(n_seq=65537), INVALID), (dict(n_tok=-1), INVALID), (dict(width=0), INVALID),
             (dict(stride=3), INVALID), (dict(reserved=1), INVALID), (dict(table=P + 2), MISALIGNED),
             (dict(past=P + 1), MISALIGNED), (dict(q_start=P + 2), MISALIGNED)]


@pytest.mark.parametrize("which,kw,want", [("c", *x) for x in BAD_CACHE] + [("b", *x) for x in BAD_BATCH])
def test_cache_and_batch_fields(L, which, kw, want):
    c, b = (cache(**kw), batch()) if which == "c" else (cache(), batch(**kw))
    big = dict(klt=10 ** 6, vlt=10 ** 6, klh=300, vlh=300, qlh=300, olh=300)
    assert append(L, c, b, rot=0, **big) == want
    assert attend(L, c, b, heads=c.n_kv_heads or 1, qlh=300, olh=300) == want
    assert L.rf_kv_read(ref(c), ref(b), P, P, 0, None) == want
    assert L.rf_attention_workspace_bytes(ref(c), ref(b), rf.F32, c.n_kv_heads or 1, 0, 0) == 0


def test_null_cache_or_batch(L):
    for c, b in ((None, batch()), (cache(), None)):
        assert append(L, c, b) == attend(L, c, b) == L.rf_kv_read(ref(c), ref(b), P, P, 0, None) == INVALID


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(dtype=12), UNSUPPORTED), (dict(rot=4), INVALID), (dict(rot=72), INVALID), (dict(rot=-8), INVALID),
    (dict(cos=None), INVALID), (dict(sin=None), INVALID), (dict(n_pos=0), INVALID),
    (dict(rot=0, cos=None, sin=None, n_pos=0), OK), (dict(style=2), INVALID), (dict(flags=4), INVALID),
    (dict(qo=None), INVALID), (dict(heads=0), INVALID), (dict(qlh=63), INVALID), (dict(olt=63), INVALID),
    (dict(q=None, qo=None, heads=0), OK), (dict(k=P + 2), MISALIGNED), (dict(cos=P + 4), MISALIGNED),
    (dict(heads=4097), TOO_LARGE)])
def test_append_arguments(L, kw, want):
    assert append(L, cache(), batch(), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(klt=63), INVALID), (dict(klh=63), INVALID),
    (dict(vlt=63), INVALID), (dict(vlh=63), INVALID)])
def test_append_arguments_with_tokens(L, kw, want):
    assert append(L, cache(), batch(n_tok=1), **kw) == want


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(dtype=2), UNSUPPORTED), (dict(heads=3), INVALID), (dict(heads=0), INVALID),
    (dict(window=-1), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(max_len=-1), INVALID), (dict(flags=8), INVALID), (dict(q=P + 2), MISALIGNED),
    (dict(q=P + 2, dtype=rf.F16), OK), (dict(sinks=P + 2), MISALIGNED), (dict(ws=P + 128), MISALIGNED),
    (dict(heads=4098), TOO_LARGE)])
def test_attention_arguments(L, kw, want):
    assert attend(L, cache(), batch(), **kw) == want


@pytest.mark.parametrize("kw", [dict(q=None), dict(out=None), dict(qlt=63), dict(qlh=63), dict(olt=63), dict(olh=63)])
def test_attention_arguments_with_tokens(L, kw):
    assert attend(L, cache(), batch(n_tok=1), **kw) == INVALID


def test_read_arguments(L):
    c, b = cache(), batch(n_tok=1)
    assert L.rf_kv_read(ref(c), ref(b), None, P, 0, None) == INVALID
    assert L.rf_kv_read(ref(c), ref(b), P, None, 0, None) == INVALID
    assert L.rf_kv_read(ref(c), ref(b), P + 8, P, 0, None) == MISALIGNED
    assert L.rf_kv_read(ref(c), ref(b), P, P, 2, None) == INVALID
    assert L.rf_kv_read(ref(c), ref(batch()), None, None, 0, None) == OK


def test_binding_refuses_what_is_not_a_device_tensor():
    import torch
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        rf.norm_residual(x)
    with pytest.raises(ValueError):
        rf.norm_residual(None)
    z, e = torch.zeros((2, 1, 64, 16), dtype=torch.int8), torch.zeros((2, 1, 2), dtype=torch.uint8)
    with pytest.raises(ValueError):
        rf.KVCache(z, z, e, e)
    with pytest.raises(ValueError):
        rf.KVCache(z.float(), z, e, e)
    with pytest.raises(ValueError):
        rf.KVCache(z, z, e[:, :, :1], e)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        rf.KVBatch(i.view(1, 1), i, torch.zeros(2, dtype=torch.int32), 0)
