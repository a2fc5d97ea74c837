"""Argument checks of fp32 outputs: made on the host, pointers never read."""
import ctypes

import pytest

import quantized_weight_streaming_dequant_gb300 as rf

P, BIG = 1 << 20, 1 << 50


@pytest.fixture(scope="module")
def L():
    from quantized_weight_streaming_dequant_gb300 import build
    build.build()
    return rf.lib()


def fused(L, dtype, n_tok=0, X=P, Y=P, residual=None, bytes=BIG):
    e = rf.Epilogue(None, None, residual, 64, 0, 1.0, 1.0, 0)
    return L.rf_gemm_fused(rf.Q4_0, P, None, 0, 64, 64, dtype, n_tok, X, 64, ctypes.byref(e), Y, 64, P, bytes, None)


@pytest.mark.parametrize("x", [rf.F32, rf.F16, rf.BF16])
def test_fp32_outputs_are_aligned_to_four_bytes(L, x):
    half = x != rf.F32
    assert fused(L, x | rf.Y_F32) == 0 and fused(L, x | rf.Y_F32, residual=P) == 0
    assert fused(L, x | rf.Y_F32, X=P + 2) == (0 if half else 8)
    assert fused(L, x | rf.Y_F32, Y=P + 2) == 8 and fused(L, x | rf.Y_F32, residual=P + 2) == 8
    assert fused(L, x, Y=P + 2) == (0 if half else 8)
    assert fused(L, x | rf.Y_F32, n_tok=1, bytes=64) == 1


@pytest.mark.parametrize("dtype", [rf.Y_F32 | 5, rf.Y_F32 | 512, -1, 2 * rf.Y_F32])
def test_unknown_types(L, dtype):
    assert fused(L, dtype) == 2
    assert L.rf_gemm_fused_workspace_bytes(rf.Q4_0, 64, 64, dtype, 9) == 0


def test_workspace_of_fp32_outputs(L):
    for n_tok in (1, 9, 300):
        for fmt in (rf.Q4_0, rf.MXFP4):
            assert L.rf_gemm_fused_workspace_bytes(fmt, 64, 256, rf.BF16 | rf.Y_F32, n_tok) > 0
        assert L.rf_gemm_fused_workspace_bytes(rf.Q4_0, 64, 256, rf.F32 | rf.Y_F32, n_tok) == \
            L.rf_gemm_fused_workspace_bytes(rf.Q4_0, 64, 256, rf.F32, n_tok)


def test_routing_and_the_routed_ffn_have_one_type(L):
    assert L.rf_moe_tokens_workspace_bytes(rf.MXFP4, 8, 2, 96, 64, rf.BF16 | rf.Y_F32, 10) == 0
    assert L.rf_moe_route_tokens(rf.F32 | rf.Y_F32, P, 8, 9, 8, 2, P, P, P, P, P, P, BIG, None) == 2
    assert L.rf_moe_ffn_tokens(rf.MXFP4, rf.BF16 | rf.Y_F32, rf.F32, P, 8, 8, 2, 0, P, P, P, None, None, None,
                               rf.ACT_SWIGLU, 1.0, 1.0, 96, 64, P, 64, None, 0, P, 64, P, BIG, None) == 2
