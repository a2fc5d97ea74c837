"""The cases that measure the operators of a chunk of tokens through quantized weights.

Four operators, as a user of the library calls them:

  route    `rf.moe_route_tokens`: the top-k experts of each token of a chunk,
           their weights, and the chunk's rows in the order of their experts.
  grouped  `rf.gemm_grouped`: each expert's matrix times its own rows, groups of
           ragged sizes, empty ones among them.
  moe      `rf.moe_ffn_tokens`: the routed FFN of a chunk: route, gate and up with
           the activation, down, and the weighted sum over each token's experts.
  fused    `rf.gemm_fused`: a quantized matrix times a chunk with bias, activation
           (or gate and up matrix) and residual in the same pass.

With `own` false, `run` computes the same in elementary torch operations in 32
bits; with `own` true it calls the library.
"""
import math

import torch

own = False

DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
# weights in a block, its bytes
BLOCK = {"Q4_0": (32, 18), "Q8_0": (32, 34), "MXFP4": (32, 17), "Q4_K": (256, 144)}
ALPHA, LIMIT = 1.702, 7.0   # constants of the clamped SwiGLU


# ------------------------------------------------------------------ the cases
def _route(name, n_tok, experts, top_k, dtype):
    return {"name": name, "op": "route", "n_tok": n_tok, "experts": experts, "top_k": top_k, "dtype": dtype}


def _grouped(name, fmt, dtype, n_rows, groups, rows, inputs, bias):
    return {"name": name, "op": "grouped", "fmt": fmt, "dtype": dtype, "n_tok": n_rows, "groups": groups,
            "rows": rows, "inputs": inputs, "bias": bias}


def _moe(name, fmt, dtype, n_tok, experts, top_k, embd, ff, clamped, residual):
    return {"name": name, "op": "moe", "fmt": fmt, "dtype": dtype, "n_tok": n_tok, "experts": experts, "top_k": top_k,
            "embd": embd, "ff": ff, "clamped": clamped, "residual": residual}


def _fused(name, fmt, dtype, n_tok, rows, inputs, act, bias, residual):
    return {"name": name, "op": "fused", "fmt": fmt, "dtype": dtype, "n_tok": n_tok, "rows": rows, "inputs": inputs,
            "act": act, "bias": bias, "residual": residual}


def listed():
    return [
        # a few tokens in flight: latency
        _route("route_few", 5, 128, 4, "f32"),
        # a prompt, 16-bit logits (equal ones among them)
        _route("route_prompt", 8192, 128, 4, "bf16"),
        # a projection of its own for each of many groups, few rows in most and none in some
        _grouped("grouped_few", "Q8_0", "f32", 45, 64, 1408, 2048, False),
        # ragged groups of a prompt, with a bias for each group
        _grouped("grouped_prompt", "Q4_0", "f16", 5000, 24, 4000, 2080, True),
        # a decode batch through the 128-expert layer of the benchmark: nearly all weights for few rows
        _moe("moe_few", "MXFP4", "f32", 6, 128, 4, 2880, 2880, True, False),
        # a short chunk of odd length through the same layer
        _moe("moe_chunk", "MXFP4", "bf16", 77, 128, 4, 2880, 2880, True, True),
        # a prompt through the same layer
        _moe("moe_prompt", "MXFP4", "bf16", 2048, 128, 4, 2880, 2880, True, False),
        # few large experts of the dense layer's sizes
        _moe("moe_large", "Q4_0", "bf16", 1001, 8, 2, 4096, 11008, False, True),
        # just more tokens than the multi-token GEMV takes: gate and up of the dense layer
        _fused("fused_few", "Q4_0", "f32", 9, 11008, 4096, "swiglu", False, False),
        # a chunk of odd length through a biased projection
        _fused("fused_chunk", "Q4_K", "f32", 77, 4099, 4096, "gelu", True, False),
        # a prompt: gate and up of the dense layer
        _fused("fused_prompt", "Q4_0", "bf16", 2048, 11008, 4096, "swiglu", False, False),
        # and its way back into the residual stream
        _fused("fused_down", "Q8_0", "bf16", 2048, 4096, 11008, "none", False, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _inputs(rng, fmt, lo, hi):
    block = BLOCK[fmt][0]
    return max(1, _log(rng, lo, hi) // block) * block


def draw(rng):
    op = rng.choice(("route", "grouped", "moe", "moe", "fused", "fused"))
    top = work(listed()[6])
    while True:
        dtype = rng.choice(("f32", "bf16", "bf16", "f16"))
        fmt = rng.choice(("MXFP4", "MXFP4", "Q4_0", "Q8_0", "Q4_K"))
        n_tok = _log(rng, 1, 4096)
        if op == "route":
            experts = _log(rng, 2, 1024)
            c = _route("", _log(rng, 1, 8192), experts, min(experts, rng.randint(1, 8)), dtype)
            ok = c["n_tok"] * experts <= 8192 * 128
        elif op == "grouped":
            c = _grouped("", fmt, dtype, n_tok, _log(rng, 1, 128), _log(rng, 64, 8192), _inputs(rng, fmt, 64, 8192),
                         rng.random() < 0.5)
            ok = True
        elif op == "moe":
            experts = _log(rng, 2, 160)
            c = _moe("", fmt, dtype, n_tok, experts, min(experts, rng.choice((1, 2, 2, 4, 4, 6, 8))),
                     _inputs(rng, fmt, 256, 6144), _inputs(rng, fmt, 128, 11008), rng.random() < 0.5, rng.random() < 0.5)
            ok = True
        else:
            c = _fused("", fmt, dtype, n_tok, _log(rng, 64, 16384), _inputs(rng, fmt, 64, 16384),
                       rng.choice(("none", "silu", "gelu", "swiglu", "clamped")), rng.random() < 0.5, rng.random() < 0.5)
            ok = True
        if op != "route":
            w = work(c)
            held = sum(r * i * g for r, i, g in _matrices(c))   # what the plain form holds in 32 bits
            ok = w["flops"] <= top["flops"] and w["bytes"] <= top["bytes"] and held <= 3 * 128 * 2880 * 2880
        if ok:
            del c["name"]
            return c


def _matrices(case):
    """(rows, inputs, copies) of each weight tensor."""
    if case["op"] == "moe":
        e = case["experts"]
        return [(case["ff"], case["embd"], e), (case["ff"], case["embd"], e), (case["embd"], case["ff"], e)]
    n = case.get("groups", 1)
    return [(case["rows"], case["inputs"], n)] * (2 if case.get("act") in ("swiglu", "clamped") else 1)


def work(case):
    t, b = case["n_tok"], SIZE[case["dtype"]]
    if case["op"] == "route":
        e, k = case["experts"], case["top_k"]
        return {"bytes": t * e * b + 4 * t * k * 4 + 4 * (e + 1), "flops": t * e * (k + 1)}
    block, size = BLOCK[case["fmt"]]
    weights = sum(r * (i // block) * size * n for r, i, n in _matrices(case))
    product = sum(2 * r * i for r, i, _ in _matrices(case))
    if case["op"] == "moe":
        e, k = case["experts"], case["top_k"]
        hit = 1 - (1 - k / e) ** t                                 # share of the experts that get a token
        return {"bytes": weights * hit + t * (case["embd"] * b * (2 + case["residual"]) + e * b), "flops": t * k * product}
    if case["op"] == "grouped":
        g = case["groups"]
        hit = sum(n > 0 for n in _sizes(case)) / g
        return {"bytes": weights * hit + t * (case["rows"] + case["inputs"]) * b + 4 * g * (1 + case["rows"] * case["bias"]),
                "flops": t * product}
    return {"bytes": weights + t * (case["inputs"] + case["rows"] * (1 + case["residual"])) * b
            + 4 * case["rows"] * case["bias"] * len(_matrices(case)), "flops": t * product}


def _sizes(case):
    """Rows of each group of a "grouped" case: ragged, every seventh group empty."""
    g, n = case["groups"], case["n_tok"]
    share = [0 if i % 7 == 3 else 1 + (i * 5) % 11 for i in range(g)]
    total, sizes, done, seen = sum(share), [], 0, 0
    for s in share:
        seen += s
        upto = n * seen // total
        sizes.append(upto - done)
        done = upto
    return sizes


# ------------------------------------------------------------------ the inputs
def _weights(g, fmt, rows, inputs, n):
    """Random blocks, as files of quantized weights hold them: (n * rows, bytes)."""
    block, size = BLOCK[fmt]
    w = torch.randint(0, 256, (n * rows, inputs // block, size), generator=g, device="cuda", dtype=torch.uint8)
    if fmt == "MXFP4":
        w[..., 0] = torch.randint(119, 126, w.shape[:2], generator=g, device="cuda", dtype=torch.uint8)
        return w.flatten(1)
    lo, hi, n_scale = {"Q4_0": (1e-3, 2e-2, 1), "Q8_0": (1e-3, 1e-2, 1), "Q4_K": (1e-4, 1e-3, 2)}[fmt]
    d = lo + (hi - lo) * torch.rand((*w.shape[:2], n_scale), generator=g, device="cuda")
    w[..., :2 * n_scale] = d.half().view(torch.uint8)
    return w.flatten(1)


def _randn(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, t = DTYPE[case["dtype"]], case["n_tok"]
    s = {"case": case}
    if case["op"] in ("route", "moe"):
        # some experts are more popular than others
        e = case["experts"]
        s["logits"] = (0.5 * _randn(g, (e,)) + _randn(g, (t, e))).to(dt)
    if case["op"] == "route":
        return s
    m = _matrices(case)
    s["w"] = [_weights(g, case["fmt"], *x) for x in m]
    s["x"] = _randn(g, (t, m[0][1]), dt)
    if case["op"] == "grouped":
        starts = [0]
        for n in _sizes(case):
            starts.append(starts[-1] + n)
        s["offsets"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    biased = case["clamped"] if case["op"] == "moe" else case["bias"]
    s["bias"] = [_randn(g, (n, r)) if biased else None for r, _, n in m]
    s["residual"] = _randn(g, (t, m[-1][0]), dt) if case.get("residual") else None
    return s


# ------------------------------------------------------------- the plain forms
def _plain_route(logits, top_k):
    x = logits.float()
    x = torch.where(x.isnan(), torch.full_like(x, -math.inf), x)
    v, at = torch.sort(x, dim=1, descending=True, stable=True)
    e = (v[:, :top_k] - v[:, :1]).exp()
    idx = at[:, :top_k].to(torch.int32)
    order = torch.argsort(idx.flatten(), stable=True)
    counts = torch.bincount(idx.flatten(), minlength=logits.shape[1])
    offsets = torch.cat((torch.zeros_like(counts[:1]), counts.cumsum(0)))
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    return idx, e / e.sum(1, keepdim=True), offsets.to(torch.int32), order.to(torch.int32), place.to(torch.int32)


def _half(b):
    return b.contiguous().view(torch.float16).float()


def _plain_values(fmt, w):
    """(matrix rows, inputs) in 32 bits."""
    b = w.unflatten(1, (-1, BLOCK[fmt][1]))
    if fmt == "Q8_0":
        return (b[..., 2:].view(torch.int8).float() * _half(b[..., :2])).flatten(1)
    if fmt == "Q4_K":
        sc, q = b[..., 4:16], b[..., 16:].unflatten(2, (4, 32))
        low = torch.cat((sc[..., :4] & 63, (sc[..., 8:] & 15) | (sc[..., :4] >> 6 << 4)), -1).float()
        least = torch.cat((sc[..., 4:8] & 63, (sc[..., 8:] >> 4) | (sc[..., 4:8] >> 6 << 4)), -1).float()
        q = torch.stack((q & 15, q >> 4), 3).flatten(2, 3).float()             # (row, block, 8, 32)
        return (q * (low * _half(b[..., :2]))[..., None] - (least * _half(b[..., 2:4]))[..., None]).flatten(1)
    start = 1 if fmt == "MXFP4" else 2
    q = torch.cat((b[..., start:] & 15, b[..., start:] >> 4), -1)
    if fmt == "Q4_0":
        return ((q.float() - 8) * _half(b[..., :2])).flatten(1)
    size = q & 7
    exp = (size >> 1).float()
    v = torch.where(exp == 0, 0.5 * (size & 1), torch.exp2(exp - 1) * (1 + 0.5 * (size & 1)))
    return (torch.where(q > 7, -v, v) * torch.exp2(b[..., :1].float() - 127)).flatten(1)


def _plain_act(act, z, u):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == "swiglu":
        return z / (1 + torch.exp(-z)) * u
    if act == "clamped":
        z, u = z.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
        return z / (1 + torch.exp(-ALPHA * z)) * (u + 1)
    return z


def _plain_groups(fmt, w, n, x, at, bias):
    """x (group, row, inputs) through each group's matrix; the rows at `at`."""
    y = torch.bmm(x, _plain_values(fmt, w).unflatten(0, (n, -1)).transpose(1, 2))
    if bias is not None:
        y += bias[:, None]
    return y[at]


def _spread(x, offsets, most):
    """Sorted rows as (group, row, ...) and their places there."""
    row = torch.arange(x.shape[0], device="cuda")
    group = (row[:, None] >= offsets[None, 1:]).sum(1)
    at = (group, row - offsets[group])
    padded = torch.zeros((offsets.numel() - 1, most, x.shape[1]), device="cuda")
    padded[at] = x
    return padded, at


def _plain_moe(s):
    case = s["case"]
    e, k, fmt = case["experts"], case["top_k"], case["fmt"]
    _, weight, offsets, order, place = _plain_route(s["logits"], k)
    offsets = offsets.long()
    most = int((offsets[1:] - offsets[:-1]).max())
    x, at = _spread(s["x"].float()[order.long() // k], offsets, most)
    g = _plain_groups(fmt, s["w"][0], e, x, at, s["bias"][0])
    u = _plain_groups(fmt, s["w"][1], e, x, at, s["bias"][1])
    h, at = _spread(_plain_act("clamped" if case["clamped"] else "swiglu", g, u), offsets, most)
    d = _plain_groups(fmt, s["w"][2], e, h, at, s["bias"][2])
    y = (d[place.long()].unflatten(0, (-1, k)) * weight[..., None]).sum(1)
    return [(y if s["residual"] is None else s["residual"].float() + y).to(s["x"].dtype)]


def _plain_grouped(s):
    offsets = s["offsets"].long()
    x, at = _spread(s["x"].float(), offsets, max(_sizes(s["case"])))
    return [_plain_groups(s["case"]["fmt"], s["w"][0], s["case"]["groups"], x, at, s["bias"][0]).to(s["x"].dtype)]


def _plain_fused(s):
    x, z = s["x"].float(), []
    for w, bias in zip(s["w"], s["bias"]):
        y = x @ _plain_values(s["case"]["fmt"], w).t()
        z.append(y if bias is None else y + bias)
    y = _plain_act(s["case"]["act"], z[0], z[-1])
    return [(y if s["residual"] is None else s["residual"].float() + y).to(s["x"].dtype)]


# ------------------------------------------------------------------- one pass
def _handles(s):
    """What a user's program makes once and keeps: the format's number and the workspace."""
    import quantized_weight_streaming_dequant_gb300 as rf
    case = s["case"]
    h = {"rf": rf}
    if case["op"] == "route":
        return h
    h["fmt"] = rf.FORMATS[case["fmt"]]
    if case["op"] == "moe":
        h["workspace"] = rf.moe_tokens_workspace(h["fmt"], case["experts"], case["top_k"], case["ff"], case["embd"], s["x"])
    elif case["op"] == "grouped":
        h["workspace"] = rf.gemm_grouped_workspace(h["fmt"], case["groups"], case["rows"], case["inputs"], s["x"], case["n_tok"])
    else:
        h["workspace"] = rf.gemm_fused_workspace(h["fmt"], case["rows"], case["inputs"], s["x"])
        h["act"] = {"none": rf.ACT_NONE, "silu": rf.ACT_SILU, "gelu": rf.ACT_GELU, "swiglu": rf.ACT_SWIGLU,
                    "clamped": rf.ACT_SWIGLU_CLAMPED}[case["act"]]
    return h


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "route":
            return list(_plain_route(s["logits"], case["top_k"]))
        return {"grouped": _plain_grouped, "moe": _plain_moe, "fused": _plain_fused}[op](s)
    if "handles" not in s:
        s["handles"] = _handles(s)
    h = s["handles"]
    rf = h["rf"]
    if op == "route":
        r = rf.moe_route_tokens(s["logits"], case["top_k"])
        return [r.idx, r.w, r.offsets, r.order, r.place]
    if op == "grouped":
        return [rf.gemm_grouped(h["fmt"], s["w"][0], case["rows"], case["inputs"], s["x"], s["offsets"], bias=s["bias"][0],
                                workspace=h["workspace"])]
    if op == "moe":
        more = {"alpha": ALPHA, "limit": LIMIT} if case["clamped"] else {}
        return [rf.moe_ffn_tokens(h["fmt"], s["logits"], case["top_k"], *s["w"], case["ff"], case["embd"], s["x"],
                                  gate_bias=s["bias"][0], up_bias=s["bias"][1], down_bias=s["bias"][2],
                                  residual=s["residual"], workspace=h["workspace"], **more)]
    gated = len(s["w"]) == 2
    more = {"alpha": ALPHA, "limit": LIMIT} if case["act"] == "clamped" else {}
    return [rf.gemm_fused(h["fmt"], s["w"][0], 0, case["rows"], case["inputs"], s["x"], act=h["act"],
                          up=s["w"][1] if gated else None, bias=s["bias"][0], up_bias=s["bias"][1] if gated else None,
                          residual=s["residual"], workspace=h["workspace"], **more)]


# ------------------------------------------------------------ in 64 bits, apart
def _exact_matrix(fmt, raw, inputs):
    """One matrix of raw blocks in 64 bits, from tables of what each byte holds."""
    size = BLOCK[fmt][1]
    raw = raw.reshape(raw.shape[0], -1, size)
    table = lambda v: torch.tensor(v, dtype=torch.float64, device="cuda")  # noqa: E731
    scale = lambda lo: raw[:, :, lo:lo + 2].clone().view(torch.float16).double()  # noqa: E731
    out = torch.empty((raw.shape[0], raw.shape[1], BLOCK[fmt][0]), dtype=torch.float64, device="cuda")
    if fmt == "Q8_0":
        out[:] = table([v - 256 if v > 127 else v for v in range(256)])[raw[:, :, 2:].long()] * scale(0)
    elif fmt in ("Q4_0", "MXFP4"):
        if fmt == "Q4_0":
            code, unit, first = [n - 8 for n in range(16)], scale(0), 2
        else:
            code = [0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6]
            unit, first = table([2.0 ** (v - 127) for v in range(256)])[raw[:, :, :1].long()], 1
        both = table([[code[v % 16], code[v // 16]] for v in range(256)])[raw[:, :, first:].long()]
        out[:, :, :16], out[:, :, 16:] = both[..., 0] * unit, both[..., 1] * unit
    else:
        field = raw[:, :, 4:16].long()
        for j in range(8):
            if j < 4:
                mul, sub = field[:, :, j] % 64, field[:, :, j + 4] % 64
            else:
                mul = field[:, :, j + 4] % 16 + field[:, :, j - 4] // 64 * 16
                sub = field[:, :, j + 4] // 16 + field[:, :, j] // 64 * 16
            at = 16 + 32 * (j // 2)
            code = raw[:, :, at:at + 32].long()
            code = code // 16 if j % 2 else code % 16
            out[:, :, 32 * j:32 * j + 32] = (scale(0) * mul[..., None]) * code - scale(2) * sub[..., None]
    return out.reshape(raw.shape[0], inputs)


def _exact_activation(act, z, u):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * (1 - torch.special.erfc(z / math.sqrt(2)) / 2)
    if act == "swiglu":
        return z * torch.sigmoid(z) * u
    if act == "clamped":
        z = torch.minimum(z, torch.full_like(z, LIMIT))
        u = torch.maximum(torch.minimum(u, torch.full_like(u, LIMIT)), torch.full_like(u, -LIMIT))
        return z * torch.sigmoid(ALPHA * z) * (u + 1)
    return z


def _exact_picks(logits, top_k):
    """The experts of each token, best first, and their weights, one pick at a time."""
    left = logits.double().clone()
    left[left.isnan()] = -math.inf
    here = torch.arange(left.shape[1], device="cuda")
    free = torch.ones_like(left, dtype=torch.bool)
    idx, val = [], []
    for _ in range(top_k):
        best = left.masked_fill(~free, -math.inf).amax(1, keepdim=True)
        i = torch.where(free & (left == best), here, left.shape[1]).amin(1)     # ties: the lowest
        idx.append(i)
        val.append(left.gather(1, i[:, None])[:, 0])
        free[torch.arange(left.shape[0], device="cuda"), i] = False
    return torch.stack(idx, 1), torch.softmax(torch.stack(val, 1), 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return [None, _exact_picks(s["logits"], case["top_k"])[1], None, None, None]
    fmt, x, n = case["fmt"], s["x"].double(), _matrices(case)

    def through(i, group, rows):
        r, c, _ = n[i]
        y = rows @ _exact_matrix(fmt, s["w"][i][group * r:(group + 1) * r], c).t()
        return y if s["bias"][i] is None else y + s["bias"][i][group].double()

    if case["op"] == "fused":
        z = [through(i, 0, x) for i in range(len(n))]
        y = _exact_activation(case["act"], z[0], z[-1])
    elif case["op"] == "grouped":
        first, parts = 0, []
        for i, size in enumerate(_sizes(case)):
            parts.append(through(0, i, x[first:first + size]))
            first += size
        y = torch.cat(parts)
    else:
        idx, weight = _exact_picks(s["logits"], case["top_k"])
        y = torch.zeros((case["n_tok"], case["embd"]), dtype=torch.float64, device="cuda")
        for i in range(case["experts"]):
            tok, slot = (idx == i).nonzero(as_tuple=True)
            if tok.numel():
                h = _exact_activation("clamped" if case["clamped"] else "swiglu", through(0, i, x[tok]), through(1, i, x[tok]))
                y[tok] += weight[tok, slot][:, None] * through(2, i, h)
    return [y if s["residual"] is None else y + s["residual"].double()]
