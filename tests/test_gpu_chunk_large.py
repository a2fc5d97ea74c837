"""The chunk operators at the ends of their ranges: tensors of more than 2^31
elements, tens of thousands of groups, millions of tokens to route, graphs that
share a workspace, and a first call that is captured."""
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

import quantized_weight_streaming_dequant_gb300 as rf
from chunk_helpers import check, randn, raw, reference
from oracle import chunk as oc

pytestmark = pytest.mark.gpu
ROOT = Path(__file__).resolve().parent.parent


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_weight_streaming_dequant_gb300 import build
    build.build()
    yield
    assert rf.device_status() == rf.OK
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("n_tok,rows,in_dim", [(70016, 32768, 64), (33000, 70, 65536)])
def test_more_than_2_to_31_elements(n_tok, rows, in_dim):
    """Of Y, and of X (whose images then are as large)."""
    W, w = raw(rf.MXFP4, 1, rows, in_dim, 1)
    x = torch.randn((n_tok, in_dim), generator=gen(1), device="cuda", dtype=torch.bfloat16)
    res = torch.randn((n_tok, 1), generator=gen(2), device="cuda").to(torch.bfloat16).expand(n_tok, rows).contiguous()
    got = rf.gemm_fused(rf.MXFP4, W, 0, rows, in_dim, x, residual=res)
    at = [0, 1, n_tok // 2, n_tok - 200, n_tok - 2, n_tok - 1]
    y, b = reference(rf.MXFP4, "bfloat16", w[0], x[at].double().cpu().numpy(), residual=res[at].double().cpu().numpy())
    check(got[at], y, b, "bfloat16")


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_as_many_groups_as_there_may_be(dtype):
    n, rows, in_dim = 65536, 3, 64
    rng = np.random.default_rng(1)
    sizes = rng.integers(0, 3, n)
    offsets = np.concatenate([[0], np.cumsum(sizes)])
    W, w = raw(rf.MXFP4, n, rows, in_dim, 2)
    x, xv = randn(rng, (int(offsets[-1]), in_dim), dtype)
    got = rf.gemm_grouped(rf.MXFP4, W, rows, in_dim, x, torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    group = np.repeat(np.arange(n), sizes)
    y = np.einsum("ni,nri->nr", xv, w[group])
    from chunk_helpers import product_bound
    a = np.abs(w[group])
    check(got, y, product_bound(rf.MXFP4, dtype, in_dim, np.einsum("ni,nri->nr", np.abs(xv), a), a.sum(2),
                                np.abs(xv).sum(1)[:, None], np.abs(xv).max(1)[:, None]) + 2.0 ** -22 * np.abs(y), dtype)


@pytest.mark.parametrize("n_tok,n_expert,k", [(9_000_000, 3, 2), (8_388_481, 1, 1), (400_000, 300, 8)])
def test_routing_of_millions_of_tokens(n_tok, n_expert, k):
    """Runs of 65,535 tokens, all of which may pick one expert."""
    x = torch.randint(-4, 5, (n_tok, n_expert), generator=gen(3), device="cuda").float()
    x[:200_000, 0] = 9.0
    r = rf.moe_route_tokens(x, k)
    v, idx = torch.sort(x, dim=1, descending=True, stable=True)
    idx = idx[:, :k]
    assert torch.equal(r.idx.long(), idx)
    flat = idx.flatten()
    counts = torch.bincount(flat, minlength=n_expert)
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    assert torch.equal(r.offsets.long(), offsets)
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(r.order.long(), order)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device="cuda")
    assert torch.equal(r.place.long(), place)
    w = torch.softmax(v[:, :k].double(), 1)
    assert ((r.w.double() - w).abs() <= (k + 6) * 2.0 ** -24 * w).all()


def test_two_graphs_that_share_a_workspace():
    rng = np.random.default_rng(4)
    E, k, ff, embd = 6, 2, 256, 320
    G, U = (raw(rf.MXFP4, E, ff, embd, s)[0] for s in (1, 2))
    D, _ = raw(rf.MXFP4, E, embd, ff, 3)
    x, _ = randn(rng, (90, embd), "bfloat16")
    logits, _ = randn(rng, (90, E), "float32")
    space = rf.moe_tokens_workspace(rf.MXFP4, E, k, ff, embd, x)
    graphs, outs, wants = [], [], []
    for n in (90, 7):
        wants.append(rf.moe_ffn_tokens(rf.MXFP4, logits[:n], k, G, U, D, ff, embd, x[:n]))
        outs.append(torch.empty_like(wants[-1]))
    torch.cuda.synchronize()
    for n, out in zip((90, 7), outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            rf.moe_ffn_tokens(rf.MXFP4, logits[:n], k, G, U, D, ff, embd, x[:n], out, workspace=space)
    for i in (0, 1, 1, 0, 1, 0, 0):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], wants[i])


COLD = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import quantized_weight_streaming_dequant_gb300 as rf
import numpy as np
from chunk_helpers import randn, raw
rng = np.random.default_rng(5)
E, k, ff, embd, n = 6, 2, 4096 + 256, 512, {n}
G, U = (raw(rf.Q4_0, E, ff, embd, s)[0] for s in (1, 2))
D = raw(rf.Q4_0, E, embd, ff, 3)[0]
x = randn(rng, (n, embd), {dtype!r})[0]
logits = randn(rng, (n, E), "float32")[0]
out = torch.zeros_like(x)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    rf.moe_ffn_tokens(rf.Q4_0, logits, k, G, U, D, ff, embd, x, out)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(out, rf.moe_ffn_tokens(rf.Q4_0, logits, k, G, U, D, ff, embd, x))
assert rf.device_status() == 0 and bool((out != 0).any())
"""


@pytest.mark.parametrize("n,dtype", [(4, "float16"), (200, "float16"), (40, "float32")])
def test_a_process_whose_first_call_is_captured(n, dtype):
    code = COLD.format(root=str(ROOT), tests=str(ROOT / "tests"), n=n, dtype=dtype)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=240)
    assert r.returncode == 0, r.stderr[-2000:]
