"""Argument checks of the chunk operators: made on the host before anything is
enqueued, so they need no GPU (the pointers are never read)."""
import ctypes

import pytest
import torch

import quantized_weight_streaming_dequant_gb300 as rf

OK, INVALID, UNSUPPORTED, MISALIGNED, TOO_LARGE = 0, 1, 2, 8, 9
P = 1 << 20   # an aligned address that is never dereferenced
BIG = 1 << 50


@pytest.fixture(scope="module")
def L():
    from quantized_weight_streaming_dequant_gb300 import build
    build.build()
    return rf.lib()


def epilogue(**kw):
    a = dict(bias=None, up_bias=None, residual=None, ldr=0, act=0, alpha=1.0, limit=1.0, reserved=0)
    a.update(kw)
    return rf.Epilogue(a["bias"], a["up_bias"], a["residual"], a["ldr"], a["act"], a["alpha"], a["limit"], a["reserved"])


def fused(L, e=None, **kw):
    a = dict(fmt=rf.Q4_0, W=P, up=None, r0=0, r1=64, in_dim=64, dtype=rf.F32, n_tok=0, X=P, ldx=64, Y=P, ldy=64, ws=P,
             bytes=BIG)
    a.update(kw)
    return L.rf_gemm_fused(a["fmt"], a["W"], a["up"], a["r0"], a["r1"], a["in_dim"], a["dtype"], a["n_tok"], a["X"], a["ldx"],
                           ctypes.byref(e) if e is not None else None, a["Y"], a["ldy"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(fmt=rf.Q6_K, in_dim=256, ldx=256), UNSUPPORTED), (dict(fmt=7), UNSUPPORTED), (dict(dtype=5), UNSUPPORTED),
    (dict(W=None), INVALID), (dict(n_tok=1, X=None), INVALID), (dict(n_tok=1, Y=None), INVALID), (dict(in_dim=0), INVALID),
    (dict(in_dim=48, ldx=48), INVALID), (dict(fmt=rf.Q4_K, in_dim=128, ldx=128), INVALID), (dict(r0=-1), INVALID),
    (dict(r0=3, r1=2), INVALID), (dict(n_tok=-1), INVALID), (dict(ldx=63), INVALID), (dict(ldy=63), INVALID),
    (dict(n_tok=1, ws=None), INVALID), (dict(n_tok=1, bytes=100), INVALID), (dict(n_tok=1, ws=P + 16), MISALIGNED),
    (dict(W=P + 8), MISALIGNED), (dict(X=P + 2), MISALIGNED), (dict(X=P + 2, dtype=rf.F16), OK),
    (dict(Y=P + 1, dtype=rf.BF16), MISALIGNED), (dict(in_dim=(1 << 20) + 32, ldx=1 << 21), TOO_LARGE),
    (dict(r1=1 << 31, ldy=1 << 31), TOO_LARGE), (dict(n_tok=(1 << 30) + 1), TOO_LARGE),
    (dict(r0=5, r1=5, n_tok=3), OK), (dict(up=P), INVALID)])
def test_fused_arguments(L, kw, want):
    assert fused(L, **kw) == want


@pytest.mark.parametrize("e,kw,want", [
    (dict(act=rf.ACT_SILU, bias=P, residual=P, ldr=64), {}, OK), (dict(act=5), {}, INVALID), (dict(act=-1), {}, INVALID),
    (dict(reserved=1), {}, INVALID), (dict(act=rf.ACT_SWIGLU), {}, INVALID), (dict(act=rf.ACT_SWIGLU), dict(up=P), OK),
    (dict(act=rf.ACT_SWIGLU), dict(up=P + 8), MISALIGNED), (dict(act=rf.ACT_SILU), dict(up=P), INVALID),
    (dict(up_bias=P), {}, INVALID), (dict(act=rf.ACT_SWIGLU_CLAMPED), dict(up=P), OK),
    (dict(act=rf.ACT_SWIGLU_CLAMPED, limit=0.0), dict(up=P), INVALID),
    (dict(act=rf.ACT_SWIGLU_CLAMPED, limit=float("nan")), dict(up=P), INVALID),
    (dict(act=rf.ACT_SWIGLU_CLAMPED, limit=float("inf")), dict(up=P), OK),
    (dict(act=rf.ACT_SWIGLU_CLAMPED, alpha=float("inf")), dict(up=P), INVALID),
    (dict(act=rf.ACT_SWIGLU_CLAMPED, alpha=float("nan")), dict(up=P), INVALID),
    (dict(residual=P, ldr=63), {}, INVALID), (dict(residual=P + 2, ldr=64), {}, MISALIGNED), (dict(bias=P + 2), {}, MISALIGNED)])
def test_epilogue_arguments(L, e, kw, want):
    assert fused(L, epilogue(**e), **kw) == want


def grouped(L, **kw):
    a = dict(fmt=rf.MXFP4, W=P, up=None, n_group=3, rows=64, in_dim=64, dtype=rf.F32, X=P, ldx=64, n_x=9, offsets=P,
             order=None, per=1, n_row=0, Y=P, ldy=64, ws=P, bytes=BIG)
    a.update(kw)
    return L.rf_gemm_grouped(a["fmt"], a["W"], a["up"], a["n_group"], a["rows"], a["in_dim"], a["dtype"], a["X"], a["ldx"],
                             a["n_x"], a["offsets"], a["order"], a["per"], a["n_row"], None, a["Y"], a["ldy"], a["ws"],
                             a["bytes"], None)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(n_group=0), INVALID), (dict(n_group=65537), TOO_LARGE), (dict(rows=-1), INVALID), (dict(rows=0, n_row=4), OK),
    (dict(offsets=None), INVALID), (dict(per=0), INVALID), (dict(n_x=-1), INVALID), (dict(n_row=10), INVALID),
    (dict(n_row=9, ws=None), INVALID), (dict(n_row=9, bytes=64), INVALID), (dict(n_row=-1), INVALID),
    (dict(offsets=P + 2), MISALIGNED), (dict(order=P + 1), MISALIGNED), (dict(X=None), INVALID), (dict(X=None, n_x=0), OK),
    (dict(fmt=rf.Q6_K), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED)])
def test_grouped_arguments(L, kw, want):
    assert grouped(L, **kw) == want


def route(L, **kw):
    a = dict(dtype=rf.F32, logits=P, ld=8, n_tok=100, n_expert=8, k=2, idx=P, w=P, offsets=P, order=P, place=P, ws=P, bytes=BIG)
    a.update(kw)
    return L.rf_moe_route_tokens(a["dtype"], a["logits"], a["ld"], a["n_tok"], a["n_expert"], a["k"], a["idx"], a["w"],
                                 a["offsets"], a["order"], a["place"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=3), UNSUPPORTED), (dict(logits=None), INVALID), (dict(ld=7), INVALID), (dict(n_tok=-1), INVALID),
    (dict(n_expert=0, ld=0), INVALID), (dict(n_expert=1025, ld=1025), INVALID), (dict(k=0), INVALID), (dict(k=9, n_expert=16, ld=16), INVALID),
    (dict(k=5, n_expert=4), INVALID), (dict(idx=None), INVALID), (dict(w=None), INVALID), (dict(offsets=None), INVALID),
    (dict(order=None), INVALID), (dict(place=None), INVALID), (dict(ws=None), INVALID), (dict(bytes=8), INVALID),
    (dict(ws=P + 4), MISALIGNED), (dict(logits=P + 2), MISALIGNED), (dict(place=P + 2), MISALIGNED),
    (dict(n_tok=(1 << 29) + 1), TOO_LARGE)])
def test_route_arguments(L, kw, want):
    assert route(L, **kw) == want


def moe(L, **kw):
    a = dict(fmt=rf.MXFP4, dtype=rf.BF16, ldt=rf.F32, logits=P, ldl=8, n_expert=8, k=2, n_tok=0, gate=P, up=P, down=P, gb=None,
             ub=None, db=None, act=rf.ACT_SWIGLU, alpha=1.0, limit=1.0, ff=96, embd=64, X=P, ldx=64, res=None, ldr=0, Y=P,
             ldy=64, ws=P, bytes=BIG)
    a.update(kw)
    return L.rf_moe_ffn_tokens(a["fmt"], a["dtype"], a["ldt"], a["logits"], a["ldl"], a["n_expert"], a["k"], a["n_tok"], a["gate"],
                               a["up"], a["down"], a["gb"], a["ub"], a["db"], a["act"], a["alpha"], a["limit"], a["ff"], a["embd"],
                               a["X"], a["ldx"], a["res"], a["ldr"], a["Y"], a["ldy"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), (dict(fmt=rf.Q6_K), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED), (dict(ldt=9), UNSUPPORTED), (dict(gate=None), INVALID),
    (dict(up=None), INVALID), (dict(down=None), INVALID), (dict(act=rf.ACT_SILU), INVALID), (dict(act=rf.ACT_NONE), INVALID),
    (dict(ff=0), INVALID), (dict(ff=100), INVALID), (dict(embd=40, ldx=64), INVALID), (dict(ldx=63), INVALID), (dict(ldy=63), INVALID),
    (dict(res=P, ldr=63), INVALID), (dict(k=9, n_expert=9, ldl=9), INVALID), (dict(n_tok=1, ws=None), INVALID),
    (dict(n_tok=1, bytes=1), INVALID), (dict(n_tok=1, ws=P + 64), MISALIGNED), (dict(down=P + 8), MISALIGNED),
    (dict(db=P + 2), MISALIGNED), (dict(act=rf.ACT_SWIGLU_CLAMPED, limit=-1.0), INVALID), (dict(n_tok=1, X=None), INVALID),
    (dict(res=P + 1, ldr=64), MISALIGNED)])
def test_moe_arguments(L, kw, want):
    assert moe(L, **kw) == want


def test_workspace_sizes(L):
    assert L.rf_gemm_fused_workspace_bytes(rf.Q6_K, 64, 256, rf.F32, 4) == 0
    assert L.rf_gemm_fused_workspace_bytes(rf.Q4_0, 64, 48, rf.F32, 4) == 0
    assert L.rf_gemm_fused_workspace_bytes(rf.Q4_0, 64, 64, rf.F32, 0) == 0
    for dtype, terms in ((rf.F32, 2), (rf.BF16, 1)):
        # at least the operand images: 2 bytes a term, tokens up to 16 rows, inputs up to 64
        n = L.rf_gemm_fused_workspace_bytes(rf.MXFP4, 128, 2880, dtype, 100)
        assert n >= 100 * terms * 2880 * 2
        assert L.rf_gemm_grouped_workspace_bytes(rf.MXFP4, 5, 128, 2880, dtype, 100) >= n - 65536
    assert L.rf_moe_route_tokens_workspace_bytes(64, 128, 4) == 0
    assert L.rf_moe_route_tokens_workspace_bytes(8192, 128, 4) > 0
    assert L.rf_moe_route_tokens_workspace_bytes(8192, 1025, 4) == 0
    assert L.rf_moe_tokens_workspace_bytes(rf.MXFP4, 8, 2, 96, 64, rf.F32, 10) > 0
    assert L.rf_moe_tokens_workspace_bytes(rf.MXFP4, 8, 2, 100, 64, rf.F32, 10) == 0


def test_binding_refuses_what_the_library_cannot_see():
    """Shapes and types, before any device call."""
    with pytest.raises(rf.RFError):
        rf.gemm_fused(7, None, 0, 4, 32, torch.zeros(2, 32))
    with pytest.raises(ValueError, match="2-D CUDA"):
        rf.gemm_fused(rf.Q4_0, torch.zeros(18, dtype=torch.uint8), 0, 1, 32, torch.zeros(2, 32))
    with pytest.raises(ValueError, match="2-D CUDA"):
        rf.moe_route_tokens(torch.zeros(3, 4), 2)
