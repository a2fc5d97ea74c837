"""A workspace of the bytes stated for some number of rows serves every call of
as many or fewer: one is allocated for the largest chunk and kept."""
import numpy as np
import pytest

import quantized_weight_streaming_dequant_gb300 as rf

FMTS = [rf.MXFP4, rf.Q4_0, rf.Q8_0, rf.Q4_K]
TYPES = [rf.F32, rf.F16, rf.BF16, rf.BF16 | rf.Y_F32]


@pytest.fixture(scope="module")
def L():
    from quantized_weight_streaming_dequant_gb300 import build
    build.build()
    return rf.lib()


def grows(sizes):
    return all(b >= a > 0 for a, b in zip(sizes, sizes[1:]))


SHAPES = [(4096, 4096), (11008, 4096), (4096, 11008), (2880, 2816), (16384, 1024), (64, 16384 + 256), (300, 256), (100000, 1024)]


def all_grow(L):
    upto = list(range(1, 700)) + [1000, 1001, 2048, 4000, 4096, 4097, 8192, 100000]
    for fmt in FMTS:
        for dtype in TYPES:
            for rows, k in SHAPES:
                assert grows([L.rf_gemm_fused_workspace_bytes(fmt, rows, k, dtype, n) for n in upto]), (fmt, dtype, rows, k)
        for groups in (2, 7, 64, 1000):
            assert grows([L.rf_gemm_grouped_workspace_bytes(fmt, groups, 300, 2816, rf.F16, n) for n in upto]), (fmt, groups)
            assert grows([L.rf_gemm_grouped_workspace_bytes(fmt, groups, 1408, 2048, rf.F32, n) for n in upto]), (fmt, groups)
        for dtype in (rf.F32, rf.BF16):
            assert grows([L.rf_moe_tokens_workspace_bytes(fmt, 12, 4, 2816, 2048, dtype, n) for n in upto]), (fmt, dtype)


def test_stated_bytes_grow_with_the_rows(L):
    all_grow(L)


def test_routing_bytes_grow_with_the_tokens(L):
    upto = list(range(65, 9000)) + [10 ** 5, 10 ** 6, 128 * 65535, 128 * 65535 + 1, 129 * 65535 + 1, 1 << 27]
    assert grows([L.rf_moe_route_tokens_workspace_bytes(n, 128, 4) for n in upto])


@pytest.mark.gpu
def test_stated_bytes_grow_with_the_rows_on_the_gpu(L):
    """(How inputs are shared out depends on the number of SMs.)"""
    all_grow(L)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_a_workspace_for_the_largest_chunk_serves_them_all(L, dtype):
    import torch
    from chunk_helpers import randn, raw
    rng = np.random.default_rng(1)
    in_dim, rows = 4096, 2880
    W, _ = raw(rf.Q4_0, 1, rows, in_dim, 1)
    x, _ = randn(rng, (600, in_dim), dtype)
    space = rf.gemm_fused_workspace(rf.Q4_0, rows, in_dim, x)
    for n in (1, 3, 8, 9, 16, 17, 40, 92, 150, 200, 257, 300, 600):
        space.fill_(255)
        got = rf.gemm_fused(rf.Q4_0, W, 0, rows, in_dim, x[:n], workspace=space)
        assert torch.equal(got, rf.gemm_fused(rf.Q4_0, W, 0, rows, in_dim, x[:n])), n
    E, k, ff, embd = 6, 2, 1024, 2048
    G, U = (raw(rf.MXFP4, E, ff, embd, s)[0] for s in (1, 2))
    D, _ = raw(rf.MXFP4, E, embd, ff, 3)
    x, _ = randn(rng, (300, embd), dtype)
    logits, _ = randn(rng, (300, E), "float32")
    space = rf.moe_tokens_workspace(rf.MXFP4, E, k, ff, embd, x)
    for n in (1, 2, 5, 12, 13, 30, 64, 65, 100, 200, 300):
        space.fill_(255)
        got = rf.moe_ffn_tokens(rf.MXFP4, logits[:n], k, G, U, D, ff, embd, x[:n], workspace=space)
        assert torch.equal(got, rf.moe_ffn_tokens(rf.MXFP4, logits[:n], k, G, U, D, ff, embd, x[:n])), n
    assert rf.device_status() == rf.OK
