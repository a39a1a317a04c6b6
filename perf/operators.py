"""The operators of a decode step around a paged KV cache: sizes, inputs, their plain form
and the calls a program makes.

  plan      kv_page_plan       pages, positions and cache slots of a step's new tokens
  rope      rope_kv_write      rotary positions of q and k, K and V written to the cache
  attn      attn_paged_decode  attention of one new token per request over the cache
  logprobs  token_logprobs     log probability, rank, entropy and top alternatives

`own` false: the plain forms, in elementary torch operations (32 bits; angles of positions
in 64).  `own` true: this package's calls.  Head counts and sizes are those of the
package's own shapes (4 KV heads of 128 with 8 query heads each; the decode chain's 6144
rows of QKV = 40 query and 4 KV heads of 128, its 152064 output rows; depth 32768) or
generic.
"""
import math

import torch

own = False

_T = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"fp32": 4.0, "fp16": 2.0, "bf16": 2.0, "q8_0": 1.0 + 2.0 / 32}


def _lib():
    import weight_streaming_warp_gb300 as wsw
    return wsw


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # a decode step of 64 running requests: one token each, some opening a new page
        {"name": "plan decode 64", "op": "plan", "requests": 64, "cached": 8192, "new": 1, "page": 16},
        # a mixed step of a large server: decoding requests and prompt chunks together
        {"name": "plan mixed 1000", "op": "plan", "requests": 1000, "cached": 4096, "new": 130, "page": 32},
        # one new token each for 64 requests, the chain's fused QKV rows in fp32
        {"name": "rope decode 64 fp32->fp16", "op": "rope", "tokens": 64, "q_heads": 40, "kv_heads": 4, "dim": 128,
         "rot": 128, "interleaved": False, "scaling": "none", "far": 32768, "x": "fp32", "cache": "fp16", "page": 16,
         "nhd": True},
        # the same step of 17 requests into q8_0 pages, half of each head rotated
        {"name": "rope decode 17 fp32->q8_0", "op": "rope", "tokens": 17, "q_heads": 32, "kv_heads": 4, "dim": 128,
         "rot": 64, "interleaved": True, "scaling": "linear", "far": 65536, "x": "fp32", "cache": "q8_0", "page": 32,
         "nhd": True},
        # a prompt of 8191 tokens in bf16, positions scaled for a long context
        {"name": "rope prompt 8191 bf16", "op": "rope", "tokens": 8191, "q_heads": 40, "kv_heads": 4, "dim": 128,
         "rot": 128, "interleaved": False, "scaling": "by_parts", "far": 131072, "x": "bf16", "cache": "bf16",
         "page": 64, "nhd": False},
        # three short requests of a model with small heads: all latency
        {"name": "attn 3 short d64", "op": "attn", "requests": 3, "longest": 301, "kv_heads": 8, "group": 4, "dim": 64,
         "q": "fp16", "cache": "fp16", "page": 16, "nhd": True, "softcap": 0.0, "window": 0, "slopes": False},
        # one request at the package's configured depth
        {"name": "attn 1 x 32768 fp16", "op": "attn", "requests": 1, "longest": 32768, "kv_heads": 4, "group": 8,
         "dim": 128, "q": "fp32", "cache": "fp16", "page": 16, "nhd": True, "softcap": 0.0, "window": 0,
         "slopes": False},
        # a ragged batch at the chain's head counts, scores capped
        {"name": "attn 64 ragged bf16 g10", "op": "attn", "requests": 64, "longest": 8192, "kv_heads": 4, "group": 10,
         "dim": 128, "q": "bf16", "cache": "bf16", "page": 64, "nhd": False, "softcap": 30.0, "window": 0,
         "slopes": False},
        # long requests over q8_0 pages, read as they are
        {"name": "attn 32 long q8_0", "op": "attn", "requests": 32, "longest": 32768, "kv_heads": 4, "group": 8,
         "dim": 128, "q": "fp32", "cache": "q8_0", "page": 32, "nhd": False, "softcap": 0.0, "window": 0,
         "slopes": False},
        # the token just sampled by one request
        {"name": "logprobs 1 x 152064", "op": "logprobs", "rows": 1, "vocab": 152064, "x": "fp32", "top": 20,
         "scale": 1.0, "masked": False},
        # a decode step of 64 requests, some tokens forbidden
        {"name": "logprobs 64 x 152064", "op": "logprobs", "rows": 64, "vocab": 152064, "x": "fp32", "top": 8,
         "scale": 1.25, "masked": True},
        # a scored prompt, an odd vocabulary in bf16
        {"name": "logprobs 2047 x 50021 bf16", "op": "logprobs", "rows": 2047, "vocab": 50021, "x": "bf16", "top": 5,
         "scale": 1.0, "masked": False},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "attn", "attn", "logprobs"])
    if op == "plan":
        requests = _spread(rng, 1, 4096)
        return {"op": op, "requests": requests, "cached": _spread(rng, 1, 32768),
                "new": _spread(rng, 1, max(1, 130000 // requests)), "page": rng.choice([1, 8, 16, 32, 64, 256])}
    if op == "rope":
        dim = rng.choice([64, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        q_heads = kv_heads * rng.choice([1, 2, 4, 5, 8, 10])
        x, cache = rng.choice([("fp32", "fp16"), ("fp32", "q8_0"), ("bf16", "bf16"), ("fp16", "fp16")])
        return {"op": op, "tokens": _spread(rng, 1, max(1, 8191 * 48 * 128 // (dim * (q_heads + 2 * kv_heads)) // 2)),
                "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
                "rot": rng.choice([dim, dim, dim // 2, dim // 4 + 8]), "interleaved": rng.random() < 0.5,
                "scaling": rng.choice(["none", "linear", "ntk", "by_parts"]), "far": _spread(rng, 1000, 1 << 20),
                "x": x, "cache": cache, "page": rng.choice([8, 16, 64]), "nhd": rng.random() < 0.5}
    if op == "attn":
        dim = rng.choice([64, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        q, cache = rng.choice([("fp32", "fp16"), ("fp32", "q8_0"), ("bf16", "bf16"), ("fp16", "fp16"),
                               ("bf16", "q8_0")])
        requests = _spread(rng, 1, 200)
        longest = _spread(rng, 1, min(65536, 32 * 32768 * 4 * 128 // (requests * kv_heads * dim)))
        return {"op": op, "requests": requests, "longest": longest, "kv_heads": kv_heads,
                "group": rng.choice([1, 2, 3, 4, 7, 8, 10, 16]), "dim": dim, "q": q, "cache": cache,
                "page": rng.choice([1, 8, 16, 32, 64, 256]), "nhd": rng.random() < 0.5,
                "softcap": rng.choice([0.0, 0.0, 30.0]), "window": rng.choice([0, 0, _spread(rng, 1, longest)]),
                "slopes": rng.random() < 0.2}
    rows = _spread(rng, 1, 2000)
    return {"op": op, "rows": rows, "vocab": _spread(rng, 1000, min(260000, 100_000_000 // rows)),
            "x": rng.choice(["fp32", "fp16", "bf16"]), "top": rng.choice([0, 1, 5, 20, 32]),
            "scale": rng.choice([1.0, 1.25, 0.7]), "masked": rng.random() < 0.4}


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(1_000_003 * seed + 17)


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int64)


def _pages(n, page):
    return (n + page - 1) // page


def prepare(case, seed):
    g = _gen(seed)
    return {"case": case, **{"plan": _prepare_plan, "rope": _prepare_rope, "attn": _prepare_attn,
                             "logprobs": _prepare_logprobs}[case["op"]](case, g)}


def _shuffled(g, n):
    return torch.randperm(n, generator=g, device="cuda").to(torch.int32)


def _table(g, lens, page, width, spare=0):
    """A block table [requests][width] over shuffled pages (-1 past each length), and the
    pages left over, `spare` of them at least."""
    need = _pages(lens, page)
    total = int(need.sum())
    ids = _shuffled(g, total + spare)
    table = torch.full((lens.numel(), width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None, :] < need[:, None]] = ids[:total]
    return table, ids[total:]


def _prepare_plan(c, g):
    n, page = c["requests"], c["page"]
    cached = _ints(g, 0, c["cached"], n)
    new = torch.full_like(cached, c["new"])
    if c["new"] > 1:  # pairs of requests with the same sum: a step's total is the scheduler's budget
        ragged = _ints(g, 0, 2 * c["new"], n // 2)
        new[: n // 2], new[n // 2: n // 2 * 2] = ragged, 2 * c["new"] - ragged
        new = new[torch.randperm(n, generator=g, device="cuda")]
    tokens = n * c["new"]
    width = _pages(c["cached"] + 2 * c["new"], page)
    table, free = _table(g, cached, page, width, spare=int(_pages(cached + new, page).sum()) + 8)
    return {"cached": cached.to(torch.int32), "new": new.to(torch.int32), "table": table, "free": free.contiguous(),
            "head": torch.zeros(1, dtype=torch.int32, device="cuda"), "tokens": tokens,
            "positions": torch.empty(tokens, dtype=torch.int32, device="cuda"),
            "slots": torch.empty(tokens, dtype=torch.int64, device="cuda"),
            "cu": torch.empty(n + 1, dtype=torch.int32, device="cuda"),
            "lens": torch.empty(n, dtype=torch.int32, device="cuda"),
            "head_out": torch.empty(1, dtype=torch.int32, device="cuda")}


def _empty_cache(c, pages):
    """k, v (and their scales) of an unused cache, in the case's layout."""
    h, d, p = c["kv_heads"], c["dim"], c["page"]
    shape = (pages, p, h) if c["nhd"] else (pages, h, p)
    if c["cache"] != "q8_0":
        return [torch.zeros(*shape, d, dtype=_T[c["cache"]], device="cuda") for _ in range(2)] + [None, None]
    return ([torch.zeros(*shape, d, dtype=torch.int8, device="cuda") for _ in range(2)]
            + [torch.zeros(*shape, d // 32, dtype=torch.float16, device="cuda") for _ in range(2)])


def _handle(c, kv):
    return _lib().PagedKV(kv[0], kv[1], kv[2], kv[3], layout="nhd" if c["nhd"] else "hnd") if own else None


def _prepare_rope(c, g):
    t, hq, h, d = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"]
    qkv = torch.randn(t, (hq + 2 * h) * d, generator=g, device="cuda").to(_T[c["x"]])
    q, k, v = qkv.view(t, hq + 2 * h, d).split([hq, h, h], 1)
    pages = _pages(t, c["page"]) + 3
    slots = torch.randperm(pages * c["page"], generator=g, device="cuda")[:t]
    s = {"q": q, "k": k, "v": v, "positions": _ints(g, 0, c["far"] - 1, t).to(torch.int32), "slots": slots,
         "kv": _empty_cache(c, pages), "out": torch.empty(t, hq, d, dtype=_T[c["x"]], device="cuda")}
    if own:
        s["handle"] = _handle(c, s["kv"])
        s["rope"] = _lib().rope_table(c["rot"], **_scaling(c))
    return s


def _scaling(c):
    if c["scaling"] == "none":
        return {}
    return {"scaling": c["scaling"], "factor": 4.0, "original": 32768}


def _lens(c, g):
    n = c["requests"]
    lens = _ints(g, 1, c["longest"], n)
    lens[0] = c["longest"]
    if n >= 8:
        lens[n // 2] = 0  # an unused row of a padded batch
    return lens


def _prepare_attn(c, g):
    n, h, d, p = c["requests"], c["kv_heads"], c["dim"], c["page"]
    lens = _lens(c, g)
    width = _pages(c["longest"], p)
    table, _ = _table(g, lens, p, width, spare=2)
    pages = int(_pages(lens, p).sum()) + 2
    kv = _empty_cache(c, pages)
    for x in kv[:2]:
        if c["cache"] == "q8_0":
            x.copy_(torch.randint(-127, 128, x.shape, generator=g, device="cuda", dtype=torch.int8))
        else:
            x.normal_(generator=g)
    for x in kv[2:]:
        if x is not None:  # blocks of 32 normal values have their largest near 2.1
            x.copy_((torch.rand(x.shape, generator=g, device="cuda") + 1.5) / 127)
    s = {"q": torch.randn(n, h * c["group"], d, generator=g, device="cuda").to(_T[c["q"]]), "kv": kv, "table": table,
         "lens": lens.to(torch.int32), "scale": 1 / math.sqrt(d), "slopes": None,
         "out": torch.empty(n, h * c["group"], d, dtype=_T[c["q"]], device="cuda"),
         "lse": torch.empty(n, h * c["group"], dtype=torch.float32, device="cuda")}
    if c["slopes"]:
        s["slopes"] = 2.0 ** (-8 * torch.arange(1, h * c["group"] + 1, device="cuda") / (h * c["group"]))
    if own:
        s["handle"] = _handle(c, kv)
        s["ws"] = torch.zeros(_lib().attn_paged_decode_workspace_bytes(n, h * c["group"], h, d), dtype=torch.uint8,
                              device="cuda")
    return s


def _prepare_logprobs(c, g):
    n, v = c["rows"], c["vocab"]
    x = torch.randn(n, v, generator=g, device="cuda").mul_(2.5)
    noise = torch.rand(n, v, generator=g, device="cuda").clamp_(min=1e-20).log_().neg_().log_().neg_()
    if c["masked"]:
        x.masked_fill_(torch.rand(n, v, generator=g, device="cuda") < 0.01, -math.inf)
    tokens = noise.add_(x).argmax(1).to(torch.int32)  # sampled from the distribution
    x = x.to(_T[c["x"]])
    s = {"logits": x, "tokens": tokens}
    if own:
        s["ws"] = torch.zeros(max(1, _lib().token_logprobs_workspace_bytes(n, v, c["top"])), dtype=torch.uint8,
                              device="cuda")
        s["out"] = _lib().token_logprobs_out(n, c["top"], device="cuda")
    return s


# -------------------------------------------------------------- one pass --

def run(state):
    return {"plan": _plan, "rope": _rope, "attn": _attn, "logprobs": _logprobs}[state["case"]["op"]](state)


def _plan(s):
    page = s["case"]["page"]
    if own:
        p = _lib().kv_page_plan(s["cached"], s["new"], s["free"], s["head"], s["table"], page, s["tokens"],
                                out=(s["positions"], s["slots"], s["cu"], s["lens"], s["head_out"]))
        return {"table": s["table"], "positions": p.positions, "slots": p.slots, "cu": p.cu, "lens": p.seq_len,
                "head": p.head}
    cached, new, table = s["cached"].long(), s["new"].long(), s["table"]
    lens = cached + new
    have, want = _pages(cached, page), _pages(lens, page)
    upto = torch.cumsum(want - have, 0)
    first = s["head"].long() + upto - (want - have)  # of each request's new pages in the free list
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    fresh = (j >= have[:, None]) & (j < want[:, None])
    at = torch.where(fresh, first[:, None] + j - have[:, None], 0)
    table.copy_(torch.where(fresh, s["free"][at], table))
    cu = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    request = torch.repeat_interleave(torch.arange(new.numel(), device=new.device), new, output_size=s["tokens"])
    positions = torch.arange(s["tokens"], device=new.device) - cu[request] + cached[request]
    slots = table[request, positions // page].long() * page + positions % page
    return {"table": table, "positions": positions.int(), "slots": slots, "cu": cu.int(), "lens": lens.int(),
            "head": (s["head"].long() + upto[-1]).int()}


def _frequencies(c):
    """Radians per position of each rotated pair, in 64 bits, and the factor on cos and sin."""
    rot = c["rot"]
    base = 10000.0 * (4.0 ** (rot / (rot - 2)) if c["scaling"] == "ntk" else 1.0)
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    if c["scaling"] == "linear":
        return f / 4, 1.0
    if c["scaling"] == "by_parts":
        keep = ((32768 * f / (2 * math.pi) - 1) / 31).clamp(0, 1)  # turns within the original context: 1 .. 32
        return f * keep + f / 4 * (1 - keep), 0.1 * math.log(4.0) + 1
    return f, 1.0


def _rotate(x, c, positions):
    f, m = _frequencies(c)
    angle = positions.double()[:, None] * f
    cos, sin = (angle.cos() * m).float()[:, None], (angle.sin() * m).float()[:, None]
    x, r = x.float(), c["rot"]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else (x[..., : r // 2], x[..., r // 2: r])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _quantized(x):
    """q8_0 codes and scales of rows of whole 32-value blocks: d = amax / 127, x / d rounded
    to the nearest, halves away from zero."""
    b = x.unflatten(-1, (-1, 32))
    d = b.abs().amax(-1) / 127
    t = b / torch.where(d == 0, 1.0, d)[..., None]
    return (torch.sign(t) * torch.floor(t.abs() + 0.5)).flatten(-2).to(torch.int8), d.half()


def _put(cache, c, slots, rows):
    page, off = slots // c["page"], slots % c["page"]
    if c["nhd"]:
        cache[page, off] = rows
    else:
        cache[page, :, off] = rows


def _values(codes, scales):
    """What q8_0 codes stand for, in fp16."""
    return (codes.float().unflatten(-1, (-1, 32)) * scales.float()[..., None]).flatten(-2).half()


def _read_back(codes, scales):
    """A whole q8_0 cache as values: the package has a call for it."""
    if not own:
        return _values(codes, scales)
    d = codes.shape[-1]
    return _lib().dequant_q8_0_kv(codes.view(-1, 1, d), scales.view(-1, 1, d // 32)).view(codes.shape)


def _rope(s):
    c, kv = s["case"], s["kv"]
    if own:
        out = _lib().rope_kv_write(s["q"], s["k"], s["v"], s["rope"], s["positions"], s["slots"], s["handle"],
                                   interleaved=c["interleaved"], out=s["out"])
    else:
        out = _rotate(s["q"], c, s["positions"]).to(s["q"].dtype)
        rows = _rotate(s["k"], c, s["positions"]), s["v"].float()
        for i in range(2):
            if c["cache"] == "q8_0":
                codes, scales = _quantized(rows[i])
                _put(kv[i], c, s["slots"], codes)
                _put(kv[2 + i], c, s["slots"], scales)
            else:
                _put(kv[i], c, s["slots"], rows[i].to(kv[i].dtype))
    if c["cache"] == "q8_0":
        return {"q": out, "k": _read_back(kv[0], kv[2]), "v": _read_back(kv[1], kv[3])}
    return {"q": out, "k": kv[0], "v": kv[1]}


def _gathered(s, i):
    """K (0) or V (1) of every request and position in fp32, [requests][kv heads][positions][dim]."""
    c, kv, at = s["case"], s["kv"], s["table"].clamp(min=0).long()
    x = kv[i][at] if c["cache"] != "q8_0" else _values(kv[i][at], kv[2 + i][at])
    x = x.transpose(2, 3) if c["nhd"] else x  # [requests][pages][heads][page][dim]
    return x.transpose(1, 2).flatten(2, 3)[:, :, : c["longest"]].float()


def _attn(s):
    c = s["case"]
    if own:
        _lib().attn_paged_decode(s["q"], s["handle"], s["table"], s["lens"], scale=s["scale"], softcap=c["softcap"],
                                 window=c["window"], slopes=s["slopes"], out=s["out"], lse=s["lse"], ws=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    n, h, group = c["requests"], c["kv_heads"], c["group"]
    q = s["q"].float().view(n, h, group, c["dim"])
    x = q @ _gathered(s, 0).transpose(2, 3) * s["scale"]
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    p = torch.arange(c["longest"], device=q.device)
    back = s["lens"].long()[:, None] - 1 - p[None, :]  # distance from the new token
    if c["slopes"]:
        x = x - s["slopes"].float().view(1, h, group, 1) * back[:, None, None, :]
    seen = (back >= 0) & (back < (c["window"] or c["longest"]))
    x = torch.where(seen[:, None, None, :], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = w.sum(-1, keepdim=True)
    out = w @ _gathered(s, 1) / torch.where(total == 0, 1.0, total)
    return {"out": out.view(n, h * group, c["dim"]).to(s["q"].dtype),
            "lse": (m + torch.log(total)).view(n, h * group)}


def _logprobs(s):
    c = s["case"]
    if own:
        r = _lib().token_logprobs(s["logits"], s["tokens"], top=c["top"], scale=c["scale"], out=s["out"], ws=s["ws"])
        return {"logprob": r.logprob, "rank": r.rank, "lse": r.lse, "entropy": r.entropy,
                **({"top_logprob": r.top_logprob, "top_id": r.top_id} if c["top"] else {})}
    raw = s["logits"].float()
    x = raw * c["scale"]
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    lse = m + torch.log(total)
    entropy = torch.log(total) - torch.where(e > 0, e * (x - m), 0.0).sum(-1, keepdim=True) / total
    t = s["tokens"].long()[:, None]
    own_x = raw.gather(1, t)
    i = torch.arange(c["vocab"], device=x.device)[None, :]
    rank = ((raw > own_x) | ((raw == own_x) & (i < t))).sum(-1)
    got = {"logprob": (x.gather(1, t) - lse)[:, 0], "rank": rank.int(), "lse": lse[:, 0], "entropy": entropy[:, 0]}
    if c["top"]:
        bits = (raw + 0.0).view(torch.int32)
        key = (bits ^ ((bits >> 31) & 0x7fffffff)).long() * 2 ** 32 + (c["vocab"] - 1 - i)  # ties: the lowest index
        best = c["vocab"] - 1 - (key.topk(c["top"], dim=-1).values & 0xffffffff)
        got |= {"top_logprob": x.gather(1, best) - lse, "top_id": best.int()}
    return got


# ------------------------------------------------------------------- work --

def work(case):
    c = case
    if c["op"] == "plan":
        n, t = c["requests"], c["requests"] * c["new"]
        # both lengths and the open page in, lengths and offsets out; a free page in and a table entry out for each
        # page opened; position and slot of each token
        return {"bytes": 20.0 * n + 8.0 * t / c["page"] + 12.0 * t, "flops": 0.0}
    if c["op"] == "rope":
        rows = c["tokens"] * c["dim"]
        x = _BYTES[c["x"]]
        return {"bytes": rows * (x * (2 * c["q_heads"] + 2 * c["kv_heads"]) + 2 * c["kv_heads"] * _BYTES[c["cache"]])
                + 12.0 * c["tokens"], "flops": 3.0 * c["tokens"] * c["rot"] * (c["q_heads"] + c["kv_heads"])}
    if c["op"] == "attn":
        n = c["requests"]
        seen = c["window"] or c["longest"]
        mean = seen - seen * seen / (2.0 * c["longest"]) if seen < c["longest"] else c["longest"] / 2.0
        positions = min(seen, c["longest"]) + max(0, n - 1) * mean  # the first is the longest, the others even
        heads = c["kv_heads"] * c["group"]
        return {"bytes": 2 * positions * c["kv_heads"] * c["dim"] * _BYTES[c["cache"]]
                + n * heads * (2 * c["dim"] * _BYTES[c["q"]] + 4) + 4 * positions / c["page"],
                "flops": 4.0 * positions * heads * c["dim"]}
    size = c["rows"] * c["vocab"]
    return {"bytes": size * _BYTES[c["x"]] + c["rows"] * (20.0 + 8.0 * c["top"]), "flops": 5.0 * size}


# ------------------------------------------------------- 64-bit definition --

def exact(case, seed):
    """What run() returns, computed in 64 bits a request or a block of rows at a time."""
    c = case
    if c["op"] == "plan":
        return None  # whole numbers only
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attn": _exact_attn, "logprobs": _exact_logprobs}[c["op"]](c, s)


def _exact_rope(c, s):
    rot, half = c["rot"], c["rot"] // 2
    freq, m = [], 1.0
    for i in range(half):
        f = 10000.0 ** (-2.0 * i / rot)
        if c["scaling"] == "ntk":
            f = (10000.0 * 4.0 ** (rot / (rot - 2.0))) ** (-2.0 * i / rot)
        elif c["scaling"] == "linear":
            f /= 4.0
        elif c["scaling"] == "by_parts":
            m = 1.0 + 0.1 * math.log(4.0)
            turns = 32768.0 * f / (2.0 * math.pi)
            part = 0.0 if turns <= 1 else 1.0 if turns >= 32 else (turns - 1) / 31
            f = (1.0 - part) * f / 4.0 + part * f
        freq.append(f)
    z = torch.polar(torch.tensor(m, dtype=torch.float64, device="cuda"),
                    s["positions"].double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda"))
    a = torch.arange(half, device="cuda") * (2 if c["interleaved"] else 1)
    b = a + (1 if c["interleaved"] else half)

    def turned(x):
        y = x.double().clone()
        w = torch.complex(y[..., a], y[..., b]) * z[:, None]
        y[..., a], y[..., b] = w.real, w.imag
        return y

    def cache(rows):
        p, h, d = c["page"], c["kv_heads"], c["dim"]
        if c["cache"] == "q8_0":
            blocks = rows.reshape(-1, 32)
            d64 = (blocks.abs().max(1).values / 127).float().double()
            code = torch.where(d64[:, None] > 0, torch.trunc(blocks / d64.clamp(min=1e-300)[:, None]
                                                             + 0.5 * blocks.sign()), 0.0)
            rows = (code * d64.half().double()[:, None]).reshape(rows.shape)
        flat = torch.zeros(s["kv"][0].shape[0] * p, h, d, dtype=torch.float64, device="cuda")
        flat[s["slots"]] = rows
        flat = flat.view(-1, p, h, d)
        return flat if c["nhd"] else flat.permute(0, 2, 1, 3).contiguous()

    return {"q": turned(s["q"]), "k": cache(turned(s["k"])), "v": cache(s["v"].double())}


def _exact_attn(c, s):
    n, h, group, d = c["requests"], c["kv_heads"], c["group"], c["dim"]
    out = torch.zeros(n, h * group, d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, h * group), -math.inf, dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    for r in range(n):
        last = lens[r]
        start = max(0, last - c["window"]) if c["window"] else 0
        if last == 0:
            continue
        p = torch.arange(start, last, device="cuda")
        page, off = s["table"][r].long()[p // c["page"]], p % c["page"]
        got = []
        for i in range(2):
            x = s["kv"][i][page, off] if c["nhd"] else s["kv"][i][page, :, off]  # [positions][heads][dim]
            if c["cache"] == "q8_0":
                f = s["kv"][2 + i][page, off] if c["nhd"] else s["kv"][2 + i][page, :, off]
                x = (x.double() * f.double().repeat_interleave(32, -1)).half()  # a cached value is binary16
            got.append(x.double())
        q = s["q"][r].double().view(h, group, d)
        x = torch.einsum("hgd,phd->hgp", q, got[0]) * s["scale"]
        if c["softcap"]:
            x = c["softcap"] * torch.tanh(x / c["softcap"])
        if c["slopes"]:
            x = x + s["slopes"].double().view(h, group, 1) * (p - (last - 1)).double()
        lse[r] = torch.logsumexp(x, -1).reshape(-1)
        out[r] = torch.einsum("hgp,phd->hgd", torch.softmax(x, -1), got[1]).reshape(-1, d)
    return {"out": out, "lse": lse}


def _exact_logprobs(c, s):
    n = c["rows"]
    got = {k: [] for k in ("logprob", "lse", "entropy", "top_logprob")}
    step = max(1, (1 << 24) // c["vocab"])
    for r in range(0, n, step):
        x = s["logits"][r:r + step].double() * c["scale"]
        lse = torch.logsumexp(x, -1, keepdim=True)
        lp = x - lse
        got["lse"].append(lse[:, 0])
        got["entropy"].append(-(lp.exp() * lp.clamp(min=-1e30)).sum(-1))
        got["logprob"].append(lp.gather(1, s["tokens"][r:r + step].long()[:, None])[:, 0])
        if c["top"]:
            got["top_logprob"].append(lp.sort(-1, descending=True).values[:, :c["top"]])
    got = {k: torch.cat(v) for k, v in got.items() if v}
    return {**got, "rank": None, **({"top_id": None} if c["top"] else {})}
