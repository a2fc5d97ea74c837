"""GPU tests of the long-chunk attention where its CTAs work through several
items each, where rows have several parts and where fp32 sums are taken out of
tensor memory; each whole call against fp64.  The layout of a call is asked
from the library, so that the cases stay on these paths."""
import numpy as np
import pytest
import torch

import quantized_weight_streaming_dequant_gb300 as rf
from attention64 import attention64
from decoder_helpers import DTYPES, TORCH, i32

pytestmark = pytest.mark.gpu

FLUSH = 16 * 128   # positions after which fp32 sums are taken out


@pytest.fixture(autouse=True)
def clean_status():
    rf.device_status()
    yield
    assert rf.device_status() == rf.OK


def setup(seed, past, new, kv, dim, page=64, k_units=(118, 123), grow=0):
    """A cache with random codes and a ragged batch over shuffled pages.  grow:
    the keys' units double every `grow` positions of a sequence."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-(p + n) // page) for p, n in zip(past, new)]
    n_pages = sum(need) + 2
    order = torch.randperm(n_pages, generator=g, device="cuda").cpu().numpy()
    table = np.zeros((len(past), max(need)), np.int32)
    codes = lambda: (30 * torch.randn((n_pages, kv, page, dim), generator=g, device="cuda")).round_().clamp_(-127, 127).to(torch.int8)  # noqa: E731
    units = lambda lo, hi: torch.randint(lo, hi, (n_pages, kv, page // 32), generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    cache = rf.KVCache(codes(), codes(), units(*k_units), units(118, 123))
    at = 0
    for s, m in enumerate(need):
        table[s, :m] = order[at:at + m]
        at += m
        if grow:
            for j in range(m):
                for b in range(page // 32):
                    cache.k_scale[int(table[s, j]), :, b] += (j * page + 32 * b) // grow
    q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    batch = rf.KVBatch(i32(table), i32(past), i32(q_start), int(q_start[-1]))
    return g, cache, batch, table, q_start


def queries(g, n_tok, heads, dim, dtype):
    return (2 * torch.randn((n_tok, heads, dim), generator=g, device="cuda")).to(TORCH[dtype])


def check(cache, batch, table, past, q_start, q, dtype, **kw):
    out = rf.attention(cache, batch, q, **{k: torch.tensor(v, device="cuda") if k == "sinks" else v for k, v in kw.items()})
    kw.pop("max_len", None)
    ref, bound = attention64(cache, table, past, q_start, q, dtype, **kw)
    err = (out.double() - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float((err / bound).max()))
    return out


def n_items(plan, new, kv):
    return sum(-(-n // plan["item_tokens"]) for n in new) * kv * plan["head_tiles"] * plan["parts"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 200])
def test_more_items_than_ctas(dtype, dim, window):
    """Ragged lengths, so that pairs of query tiles with one empty tile are
    among the items, and items of two and of sixteen position tiles."""
    past, new = [0, 500, 37, 2000, 900, 5, 130, 0], [97, 33, 500, 1, 17, 450, 64, 5]
    g, cache, batch, table, q_start = setup(dim + window, past, new, 8, dim)
    q = queries(g, batch.n_tok, 64, dim, dtype)
    plan = rf.debug_attention_plan(cache, batch, q, window=window, max_len=2001)
    assert plan["tiles"] and n_items(plan, new, 8) > 2 * plan["sms"]
    sinks = torch.linspace(-1, 2, 64).tolist() if window else None
    out = check(cache, batch, table, past, q_start, q, dtype, window=window, max_len=2001, **({"sinks": sinks} if window else {}))
    again = rf.attention(cache, batch, q, window=window, max_len=2001, sinks=None if not window else torch.tensor(sinks, device="cuda"))
    assert torch.equal(out, again)                     # whatever CTA draws which item


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_more_items_than_ctas_in_several_parts(dtype, dim):
    """Parts of the longest sequence; the others' later parts see nothing."""
    past, new = [100, 4000, 2500, 4900, 0, 700], [90, 64, 33, 3, 70, 1]
    g, cache, batch, table, q_start = setup(10 + dim, past, new, 8, dim)
    q = queries(g, batch.n_tok, 32, dim, dtype)
    plan = rf.debug_attention_plan(cache, batch, q, max_len=4903)
    assert plan["tiles"] and plan["parts"] > 1 and n_items(plan, new, 8) > plan["sms"]
    assert plan["part_positions"] > 701                # the short ones end inside their first part
    out = check(cache, batch, table, past, q_start, q, dtype, max_len=4903)
    assert torch.equal(out, rf.attention(cache, batch, q, max_len=4903))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_fp32_sums_leave_tensor_memory(dim):
    """More than two flushes a row, lengths that end between them, maxima that
    grow from one to the next, several items a CTA."""
    past, new = [3500, 5, 1200, 4400], [300, 250, 400, 263]
    g, cache, batch, table, q_start = setup(20 + dim, past, new, 8, dim, k_units=(116, 117), grow=512)
    q = queries(g, batch.n_tok, 64, dim, "float32")
    plan = rf.debug_attention_plan(cache, batch, q, max_len=4663)
    assert plan["tiles"] and plan["parts"] == 1 and plan["part_positions"] > 2 * FLUSH and n_items(plan, new, 8) > 2 * plan["sms"]
    assert all((p + n) % FLUSH > 128 for p, n in zip(past, new))
    check(cache, batch, table, past, q_start, q, "float32", max_len=4663)


@pytest.mark.parametrize("dim", [64, 128])
def test_fp32_sums_leave_tensor_memory_in_parts(dim):
    past, new = [100, 4000, 2500, 4900, 0, 700], [90, 64, 33, 3, 70, 1]
    g, cache, batch, table, q_start = setup(30 + dim, past, new, 8, dim, k_units=(116, 117), grow=512)
    q = queries(g, batch.n_tok, 64, dim, "float32")
    plan = rf.debug_attention_plan(cache, batch, q, max_len=4903)
    assert plan["tiles"] and plan["parts"] > 1 and plan["part_positions"] > FLUSH and n_items(plan, new, 8) > plan["sms"]
    check(cache, batch, table, past, q_start, q, "float32", max_len=4903)


def test_read_back_of_many_tokens():
    """Eight tokens share a CTA where there are more than eight for each SM;
    the last CTA has three."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    past, new = [33, 0], [5 * sms + 1, 3 * sms + 2]
    _, cache, batch, table, q_start = setup(40, past, new, 3, 80)
    assert batch.n_tok == 8 * sms + 3
    for got, codes, units in zip(rf.kv_read(cache, batch), (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
        for s in range(2):
            pos = past[s] + torch.arange(new[s], device="cuda")
            page = torch.as_tensor(table[s], device="cuda").long()[pos // 64]
            want = codes[page, :, pos % 64].float() * torch.exp2(units[page, :, pos % 64 // 32].float() - 127)[..., None]
            assert torch.equal(got[q_start[s]:q_start[s + 1]], want)
