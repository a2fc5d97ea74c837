"""The armed wait fault in products of the chunk operators whose first stage is
their only one, and in launches of which most CTAs find no work: whichever CTA
has the first piece withholds its copy, the launch gives up, and the next calls
give the bits of the call before."""
import numpy as np
import pytest
import torch

import quantized_weight_streaming_dequant_gb300 as rf
from chunk_helpers import DTYPES, FMTS, NAMES, randn, raw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_weight_streaming_dequant_gb300 import build
    build.build()
    yield
    assert rf.device_status() == rf.OK


def gives_up(call):
    want = call()
    assert rf.device_status() == rf.OK
    rf.debug_arm_wait_fault(1000)
    call()
    assert rf.device_status() == 6
    assert rf.device_status() == rf.OK
    for _ in range(2):
        assert torch.equal(call(), want)
    assert rf.device_status() == rf.OK


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("n_tok,inputs", [(70, 64), (70, 128), (70, 256), (300, 128), (20, 192), (3, 64), (16, 256)])
def test_few_slices(fmt, dtype, n_tok, inputs):
    """One to four slices of inputs: for some of the kernels a single stage."""
    in_dim = 256 if fmt == rf.Q4_K else inputs
    W, _ = raw(fmt, 1, 384, in_dim, 1)
    x, _ = randn(np.random.default_rng(1), (n_tok, in_dim), dtype)
    gives_up(lambda: rf.gemm_fused(fmt, W, 0, 384, in_dim, x))


@pytest.mark.parametrize("dtype", DTYPES)
def test_most_ctas_have_no_work(dtype):
    """One group of fifty has rows: a launch of many CTAs for one or two pieces."""
    n, rows, in_dim, n_row = 50, 100, 128, 4000
    W, _ = raw(rf.Q4_0, n, rows, in_dim, 1)
    x, _ = randn(np.random.default_rng(1), (n_row, in_dim), dtype)
    offsets = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    offsets[31:] = 40
    gives_up(lambda: rf.gemm_grouped(rf.Q4_0, W, rows, in_dim, x, offsets)[:40].clone())


def test_the_first_product_of_a_routed_ffn():
    rng = np.random.default_rng(2)
    E, k, ff, embd, n_tok = 12, 4, 128, 96, 70
    G, U = (raw(rf.MXFP4, E, ff, embd, s)[0] for s in (1, 2))
    D, _ = raw(rf.MXFP4, E, embd, ff, 3)
    x, _ = randn(rng, (n_tok, embd), "bfloat16")
    logits, _ = randn(rng, (n_tok, E), "float32")
    gives_up(lambda: rf.moe_ffn_tokens(rf.MXFP4, logits, k, G, U, D, ff, embd, x))
