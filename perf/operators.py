"""The cases that measure the decoder-layer operators around the projections.

Three operators, as a user of the library calls them:

  norm    `rf.norm_residual`: an optional norm of a block's output, its gate
          and scale, the residual sum and the norm that opens the next block.
  append  `rf.kv_append`: the position rotation of q and k, and k and v into
          a paged cache of 8-bit codes with one power-of-two scale for each
          32 tokens of a head; `rf.kv_read` gives the values that the cache
          then holds.
  attend  `rf.attention`: causal attention over that cache, for single tokens
          and for chunks of a prompt.

With `own` false, `run` computes the same in elementary torch operations in
32 bits; with `own` true it calls the library.
"""
import math

import torch

own = False

DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 32            # tokens that share a scale
E_LO, E_HI = 87, 167  # scale bytes: 2^-40 .. 2^40
EPS = 1e-5


# ------------------------------------------------------------------ the cases
def _norm(name, n_tok, n, dtype, post, gate):
    return {"name": name, "op": "norm", "n_tok": n_tok, "n": n, "dtype": dtype, "post": post, "gate": gate}


def _append(name, dtype, heads, kv, dim, rot, rope, page, n_seq, past, new, ragged):
    return {"name": name, "op": "append", "dtype": dtype, "heads": heads, "kv": kv, "dim": dim, "rot": rot,
            "rope": rope, "page": page, "n_seq": n_seq, "past": past, "new": new, "ragged": ragged}


def _attend(name, dtype, heads, kv, dim, page, n_seq, past, new, ragged, window, sinks):
    return {"name": name, "op": "attend", "dtype": dtype, "heads": heads, "kv": kv, "dim": dim, "page": page,
            "n_seq": n_seq, "past": past, "new": new, "ragged": ragged, "window": window, "sinks": sinks}


def listed():
    return [
        # one decode token between two blocks of the 4096-wide dense layer: latency
        _norm("norm_token", 1, 4096, "f32", False, False),
        # a small chunk of odd length, 2880 wide, with the norm after the block and its gate
        _norm("norm_chunk", 77, 2880, "bf16", True, True),
        # a long prompt, all parts
        _norm("norm_prompt", 8192, 4096, "f32", True, True),
        # one decode token into a block that already holds some: latency
        _append("append_token", "f32", 64, 8, 64, 64, "half", 64, 1, 4107, 1, False),
        # a decode batch of ragged lengths, half of each head rotated, neighbouring pairs
        _append("append_batch", "bf16", 32, 8, 128, 64, "pairs", 32, 48, 9000, 1, True),
        # a prompt
        _append("append_prompt", "f32", 32, 8, 128, 128, "half", 64, 1, 45, 8192, False),
        # one token, short context, a K and V head for each query head (the dense 4096 layer)
        _attend("attend_token_short", "f32", 32, 32, 128, 64, 1, 500, 1, False, 0, False),
        # one token, long context, four query heads to a K and V head
        _attend("attend_token_long", "f32", 32, 8, 128, 64, 1, 131071, 1, False, 0, False),
        # a decode batch of ragged lengths, eight query heads of 64 to a K and V head, with sinks
        _attend("attend_batch", "bf16", 64, 8, 64, 32, 48, 16000, 1, True, 0, True),
        # a prompt from its first token
        _attend("attend_prompt", "bf16", 32, 8, 128, 64, 1, 0, 8192, False, 0, False),
        # a later chunk of odd length against a long past, in 32 bits
        _attend("attend_chunk", "f32", 32, 8, 128, 128, 1, 32257, 511, False, 0, False),
        # ragged prompts under a sliding window, with sinks
        _attend("attend_window", "f16", 64, 8, 64, 64, 3, 1000, 4096, True, 128, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(n):
    return n + (n % 512 == 0)


def draw(rng):
    op = rng.choice(("norm", "append", "append", "attend", "attend", "attend"))
    while True:
        dtype = rng.choice(("f32", "f32", "bf16", "f16"))
        if op == "norm":
            c = _norm("", _odd(_log(rng, 1, 8192)), _odd(_log(rng, 64, 16384)), dtype,
                      rng.random() < 0.5, rng.random() < 0.5)
            top = 8192 * 4096
            ok = c["n_tok"] * c["n"] <= top
        else:
            dim = rng.choice((64, 64, 80, 112, 128, 128, 128, 256))
            kv = rng.choice((1, 2, 4, 5, 8, 8, 16, 32))
            group = rng.choice((1, 2, 4, 5, 7, 8))
            page = rng.choice((32, 64, 128, 256))
            n_seq = _log(rng, 1, 64)
            single = rng.random() < 0.5
            past = _odd(_log(rng, 1, 131072)) - 1
            new = 1 if single else _odd(_log(rng, 2, 8192))
            ragged = n_seq > 1
            if op == "append":
                rot = rng.choice((0, dim // 2, dim, dim))
                c = _append("", dtype, kv * group, kv, dim, rot, rng.choice(("half", "pairs")), page, n_seq, past,
                            new, ragged)
                most = work(listed()[5])["bytes"]
                ok = work(c)["bytes"] <= most and n_seq * (past + new) * kv * dim <= 1 << 31
            else:
                window = rng.choice((0, 0, _log(rng, 1, 4096)))
                c = _attend("", dtype, kv * group, kv, dim, page, n_seq, past, new, ragged, window,
                            rng.random() < 0.4)
                w = work(c)
                top = work(listed()[9])
                full = kv * group * n_seq * new * (past + new)   # scores of the plain form
                ok = (w["flops"] <= top["flops"] and full <= 32 * 8192 * 8192
                      and n_seq * (past + new) * kv * dim <= 1 << 30)
        if ok:
            del c["name"]
            return c


def _lengths(case):
    """Tokens already held and tokens that come, for each sequence."""
    n, past, new = case["n_seq"], case["past"], case["new"]
    if not case["ragged"]:
        return [past] * n, [new] * n
    return ([past * (2 * i + 1) // (2 * n) for i in range(n)],
            [max(1, new * (n - i) // n) for i in range(n)])


def work(case):
    b = SIZE[case["dtype"]]
    if case["op"] == "norm":
        m = case["n_tok"] * case["n"]
        return {"bytes": 4 * m * b + 4 * case["n"] * (1 + case["post"] + case["gate"]), "flops": 8 * m}
    past, new = _lengths(case)
    n_tok, dim, kv, heads = sum(new), case["dim"], case["kv"], case["heads"]
    if case["op"] == "append":
        held = sum(p % BLOCK for p in past)   # tokens of the blocks that are continued
        blocks = sum((p + n + BLOCK - 1) // BLOCK - p // BLOCK for p, n in zip(past, new))
        return {"bytes": n_tok * (2 * heads + 2 * kv) * dim * b        # q in and out, k and v
                + 2 * (n_tok + held) * kv * dim * (1 + 4)              # codes, and their values
                + 2 * blocks * kv + n_tok * case["rot"] * 4,           # scales, cos and sin
                "flops": n_tok * (heads + 2 * kv) * dim * 4}
    pairs = seen = 0
    w = case["window"]
    for p, n in zip(past, new):
        if w:
            full = max(0, min(n, w - p - 1))                           # queries that see less than the window
            pairs += full * (p + 1) + full * (full - 1) // 2 + (n - full) * w
            seen += min(p + n, w + n - 1)
        else:
            pairs += n * p + n * (n + 1) // 2
            seen += p + n
    return {"bytes": 2 * n_tok * heads * dim * b + 2 * seen * kv * dim + 2 * seen * kv // BLOCK,
            "flops": 4 * pairs * heads * dim}


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPE[case["dtype"]]
    if case["op"] == "norm":
        m, n = case["n_tok"], case["n"]
        s = {"case": case, "x": _randn(g, (m, n), dt), "residual": (3 * _randn(g, (m, n))).to(dt),
             "w": 1 + 0.2 * _randn(g, (n,)), "scale": 0.7}
        s["w_post"] = 1 + 0.2 * _randn(g, (n,)) if case["post"] else None
        s["gate"] = 0.5 + 0.3 * _randn(g, (n,)) if case["gate"] else None
        return s
    past, new = _lengths(case)
    n_seq, page, kv, dim, heads = case["n_seq"], case["page"], case["kv"], case["dim"], case["heads"]
    n_tok, most = sum(new), max(p + n for p, n in zip(past, new))
    width = (most + page - 1) // page
    n_pages = n_seq * width + 3
    table = torch.randperm(n_pages, generator=g, device="cuda")[:n_seq * width].to(torch.int32).view(n_seq, width)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    shape = (n_pages, kv, page, dim)
    codes = lambda: (30 * _randn(g, shape, torch.float16)).round_().clamp_(-127, 127).to(torch.int8)  # noqa: E731
    scales = lambda: torch.randint(121, 124, (n_pages, kv, page // BLOCK), generator=g, device="cuda",  # noqa: E731
                                   dtype=torch.uint8)
    s = {"case": case, "n_tok": n_tok, "max_len": most, "table": table, "past": i32(past), "q_start": i32(starts),
         "q": (2 * _randn(g, (n_tok, heads, dim))).to(dt)}
    if case["op"] == "attend":
        s["cache"] = (codes(), codes(), scales(), scales())
        s["sinks"] = _randn(g, (heads,)) if case["sinks"] else None
        return s
    # an empty cache but for the blocks that are continued
    s["cache"] = (torch.zeros(shape, dtype=torch.int8, device="cuda"), torch.zeros(shape, dtype=torch.int8, device="cuda"),
                  torch.zeros((n_pages, kv, page // BLOCK), dtype=torch.uint8, device="cuda"),
                  torch.zeros((n_pages, kv, page // BLOCK), dtype=torch.uint8, device="cuda"))
    first = s["past"].long() // BLOCK * BLOCK
    at = table.long()[torch.arange(n_seq, device="cuda"), first // page]
    off = (first % page)[:, None] + torch.arange(BLOCK, device="cuda")
    for held, scale in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])):
        held[at[:, None], :, off] = (30 * _randn(g, (n_seq, BLOCK, kv, dim))).round_().clamp_(-127, 127).to(torch.int8)
        scale[at, :, first % page // BLOCK] = torch.randint(119, 124, (n_seq, kv), generator=g, device="cuda",
                                                            dtype=torch.uint8)
    s["k"], s["v"] = _randn(g, (n_tok, kv, dim), dt), _randn(g, (n_tok, kv, dim), dt)
    half = case["rot"] // 2
    s["cos"] = s["sin"] = None
    if half:
        angle = torch.arange(most, device="cuda", dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half))
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    # what is read back: the continued blocks' tokens and the new ones
    s["read_past"] = first.to(torch.int32)
    lens = [p % BLOCK + n for p, n in zip(past, new)]
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    s["read_start"], s["read_tok"] = i32(starts), starts[-1]
    return s


# ------------------------------------------------------------- the plain forms
def _plain_norm(s):
    t = s["x"].float()
    if s["w_post"] is not None:
        t = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS) * s["w_post"]
    if s["gate"] is not None:
        t = t * s["gate"]
    r = s["residual"].float() + s["scale"] * t
    y = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * s["w"]
    return [r.to(s["x"].dtype), y.to(s["x"].dtype)]


def _where(q_start, past, n_tok):
    """The sequence and the position of each of n_tok tokens."""
    tok = torch.arange(n_tok, device="cuda")
    seq = (tok[:, None] >= q_start[None, 1:]).sum(1)
    return seq, past.long()[seq] + tok - q_start.long()[seq]


def _rotate(x, cos, sin, rope):
    """x: (tokens, heads, dim); cos, sin: (tokens, 1, half)."""
    half = cos.shape[-1]
    x = x.float()
    if rope == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., 2 * half:]), -1)
    a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), x[..., 2 * half:]), -1)


def _plain_append(s):
    case = s["case"]
    page, kv, dim = case["page"], case["kv"], case["dim"]
    seq, pos = _where(s["q_start"], s["past"], s["n_tok"])
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if s["cos"] is not None:
        cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
        q, k = _rotate(q, cos, sin, case["rope"]), _rotate(k, cos, sin, case["rope"])
    # the blocks that get tokens, block j of sequence i at [i, j]
    first = s["past"].long() // BLOCK
    n_blk = max((p + n + BLOCK - 1) // BLOCK - p // BLOCK for p, n in zip(*_lengths(case)))
    blk = first[:, None] + torch.arange(n_blk, device="cuda")
    end = (s["past"].long() + (s["q_start"][1:] - s["q_start"][:-1]))[:, None]
    used = blk * BLOCK < end                                                 # (seq, block)
    old = (blk * BLOCK < s["past"][:, None]) & used                          # continued ones
    at = s["table"].long().gather(1, (blk * BLOCK // page).clamp(max=s["table"].shape[1] - 1))
    sub = blk * BLOCK % page
    rows = sub[..., None] + torch.arange(BLOCK, device="cuda")
    i, j = used.nonzero(as_tuple=True)
    for x, held, scale in ((k, s["cache"][0], s["cache"][2]), (v, s["cache"][1], s["cache"][3])):
        new = torch.zeros((case["n_seq"], n_blk, BLOCK, kv, dim), device="cuda")
        new[seq, pos // BLOCK - first[seq], pos % BLOCK] = x
        there = torch.zeros((case["n_seq"], n_blk, BLOCK), dtype=torch.bool, device="cuda")
        there[seq, pos // BLOCK - first[seq], pos % BLOCK] = True
        m, e = torch.frexp(new.abs().amax((2, 4)))                           # amax = m 2^e
        e = torch.where(m == 0, torch.full_like(e, E_LO), 127 + e - 7 + (m > 127 / 128)).clamp(min=E_LO)
        e_old = scale[at, :, sub // BLOCK].int()
        e = torch.where(old[..., None], torch.maximum(e, e_old), e)          # (seq, block, head)
        was = held[at[..., None], :, rows].float()
        was = torch.round(was * torch.exp2((e_old - e).float())[:, :, None, :, None])
        code = torch.round(new * torch.exp2((127 - e).float())[:, :, None, :, None])
        code = torch.where(there[..., None, None], code, was).to(torch.int8)
        held[at[i, j][:, None], :, rows[i, j]] = code[i, j]
        scale[at[i, j], :, sub[i, j] // BLOCK] = e[i, j].to(torch.uint8)
    out = [q.to(s["q"].dtype)]
    seq, pos = _where(s["read_start"], s["read_past"], s["read_tok"])
    at = s["table"].long()[seq, pos // page]
    for held, scale in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])):
        e = scale[at, :, pos % page // BLOCK].float() - 127
        out.append(held[at, :, pos % page].float() * torch.exp2(e)[..., None])
    return out


def _values(codes, scales, table):
    """The values of each sequence's pages: (seq, head, position, dim)."""
    c, e = codes[table.long()], scales[table.long()].float() - 127           # (seq, page, head, ...)
    v = c.float().unflatten(3, (-1, BLOCK)) * torch.exp2(e)[..., None, None]
    return v.flatten(3, 4).transpose(1, 2).flatten(2, 3)


def _plain_attend(s):
    case = s["case"]
    kv, dim, n_seq = case["kv"], case["dim"], case["n_seq"]
    group, most = case["heads"] // kv, max(_lengths(case)[1])
    k, v = (_values(s["cache"][i], s["cache"][i + 2], s["table"])[:, :, :s["max_len"]] for i in (0, 1))
    seq, pos = _where(s["q_start"], s["past"], s["n_tok"])
    at = pos - s["past"].long()[seq]
    q = torch.zeros((n_seq, most, kv, group, dim), device="cuda")
    q[seq, at] = s["q"].float().unflatten(1, (kv, group))
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3)                               # (seq, kv, group * query, dim)
    score = (q @ k.transpose(2, 3)).mul_(dim ** -0.5).unflatten(2, (group, most))
    here = torch.arange(s["max_len"], device="cuda")
    last = s["past"].long()[:, None] + torch.arange(most, device="cuda")     # the newest visible position
    hidden = here > last[..., None]
    if case["window"]:
        hidden |= here <= last[..., None] - case["window"]
    score.masked_fill_(hidden[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(1, kv, group, 1, 1)
        top = torch.maximum(top, sink)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        total = total + (sink - top).exp()
    out = ((p.flatten(2, 3) @ v).unflatten(2, (group, most)) / total).permute(0, 3, 1, 2, 4)
    return out[seq, at].flatten(1, 2).to(s["q"].dtype)


# ------------------------------------------------------------------- one pass
def _handles(s):
    """What a user's program makes once and keeps: the cache and batch handles and the workspace."""
    import quantized_weight_streaming_dequant_gb300 as rf
    h = {"rf": rf, "cache": rf.KVCache(*s["cache"]), "batch": rf.KVBatch(s["table"], s["past"], s["q_start"], s["n_tok"])}
    if s["case"]["op"] == "append":
        h["read"] = rf.KVBatch(s["table"], s["read_past"], s["read_start"], s["read_tok"])
        h["rope"] = {"half": rf.ROPE_HALF, "pairs": rf.ROPE_PAIRS}[s["case"]["rope"]]
    else:
        h["workspace"] = rf.attention_workspace(h["cache"], h["batch"], s["q"], max_len=s["max_len"],
                                                window=s["case"]["window"])
    return h


def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "norm":
            return _plain_norm(s)
        return _plain_append(s) if op == "append" else [_plain_attend(s)]
    if op == "norm":
        import quantized_weight_streaming_dequant_gb300 as rf
        return list(rf.norm_residual(s["residual"], s["x"], post_weight=s["w_post"], gate=s["gate"], scale=s["scale"],
                                     weight=s["w"], eps=EPS))
    if "handles" not in s:
        s["handles"] = _handles(s)
    h = s["handles"]
    rf = h["rf"]
    if op == "append":
        q = rf.kv_append(h["cache"], h["batch"], s["k"], s["v"], q=s["q"], cos=s["cos"], sin=s["sin"], rope=h["rope"])
        return [q, *rf.kv_read(h["cache"], h["read"])]
    return [rf.attention(h["cache"], h["batch"], s["q"], window=s["case"]["window"], sinks=s["sinks"],
                         max_len=s["max_len"], workspace=h["workspace"])]


# ------------------------------------------------------------ in 64 bits, apart
def _exact_norm(s):
    n = s["x"].shape[1]
    x, r = s["x"].double(), s["residual"].double()
    if s["w_post"] is not None:
        x = s["w_post"].double() * x / torch.sqrt(EPS + x.pow(2).sum(1)[:, None] / n)
    x = s["scale"] * x * (1 if s["gate"] is None else s["gate"].double())
    r = r + x
    return [r, s["w"].double() * r / torch.sqrt(EPS + r.pow(2).sum(1)[:, None] / n)]


def _exact_turn(x, angle_cos, angle_sin, rope):
    half = angle_cos.shape[1]
    x = x.double().clone()
    pair = torch.arange(half, device="cuda")
    a, b = (pair, pair + half) if rope == "half" else (2 * pair, 2 * pair + 1)
    z = torch.complex(x[:, :, a], x[:, :, b]) * torch.complex(angle_cos.double(), angle_sin.double())[:, None]
    x[:, :, a], x[:, :, b] = z.real, z.imag
    return x


def _exact_append(s):
    case = s["case"]
    past, new = _lengths(case)
    if sum(new) / BLOCK + len(new) > 2000:
        return None
    power = torch.tensor([2.0 ** (e - 127) for e in range(256)], dtype=torch.float64, device="cuda")
    q, ks, vs, t0 = [], [], [], 0
    for i, (p, n) in enumerate(zip(past, new)):
        q_i, k_i, v_i = (s[x][t0:t0 + n].double() for x in "qkv")
        if s["cos"] is not None:
            c, d = s["cos"][p:p + n], s["sin"][p:p + n]
            q_i, k_i = _exact_turn(q_i, c, d, case["rope"]), _exact_turn(k_i, c, d, case["rope"])
        q.append(q_i)
        for x, held, scale, got in ((k_i, s["cache"][0], s["cache"][2], ks), (v_i, s["cache"][1], s["cache"][3], vs)):
            at = p
            while at < p + n:
                b0 = at // BLOCK * BLOCK
                stop = min(b0 + BLOCK, p + n)
                page, sub = int(s["table"][i, b0 // case["page"]]), b0 % case["page"]
                part = x[at - p:stop - p]
                # the smallest power of two that keeps the codes within 127
                byte = E_LO + (part.abs().amax((0, 2))[:, None] > 127 * power[E_LO:E_HI + 1]).sum(1)
                if at > b0:
                    was = scale[page, :, sub // BLOCK].long()
                    byte = torch.maximum(byte, was)
                    old = held[page, :, sub:sub + at - b0].double().transpose(0, 1)
                    got.append((old * power[was - byte + 127][:, None]).round() * power[byte][:, None])
                got.append((part / power[byte][:, None]).round() * power[byte][:, None])
                at = stop
        t0 += n
    return [torch.cat(q), torch.cat(ks), torch.cat(vs)]


def _exact_attend(s):
    case = s["case"]
    past, new = _lengths(case)
    kv, dim, page = case["kv"], case["dim"], case["page"]
    group = case["heads"] // kv
    out = torch.empty((s["n_tok"], case["heads"], dim), dtype=torch.float64, device="cuda")
    t0 = 0
    for i, (p, n) in enumerate(zip(past, new)):
        pages = s["table"][i, :(p + n + page - 1) // page].long()
        for h in range(kv):
            k, v = ((c[pages, h].double() * 2.0 ** (e[pages, h].double() - 127).repeat_interleave(BLOCK, 1)[..., None])
                    .reshape(-1, dim)[:p + n] for c, e in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])))
            for a in range(0, n, 2048):
                b = min(n, a + 2048)
                lo = max(0, p + a + 1 - case["window"]) if case["window"] else 0
                hi = p + b
                x = s["q"][t0 + a:t0 + b, h * group:(h + 1) * group].double() / math.sqrt(dim)
                z = torch.einsum("tgd,ld->tgl", x, k[lo:hi])
                row, col = torch.arange(p + a, p + b, device="cuda")[:, None], torch.arange(lo, hi, device="cuda")
                see = col <= row
                if case["window"]:
                    see &= col > row - case["window"]
                z = torch.where(see[:, None], z, -math.inf)
                if s["sinks"] is not None:
                    z = torch.cat((z, s["sinks"].double()[h * group:(h + 1) * group].expand(b - a, group)[..., None]), -1)
                w = torch.softmax(z, -1)[..., :hi - lo]
                out[t0 + a:t0 + b, h * group:(h + 1) * group] = torch.einsum("tgl,ld->tgd", w, v[lo:hi])
        t0 += n
    return [out]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)
