"""The operators of a step in which several rows continue one prompt (beams, parallel samples,
a shared system prompt) over a paged KV cache: sizes, inputs, their plain form and the calls a
program makes.

  beam     beam_select                   the next beams from all beams' logits
  fork     kv_page_fork + kv_page_copy   block table rows of the survivors' children, and the copies of
                                         partly filled last pages in every layer
  compact  kv_page_compact               pages that no row lists any more freed, the others moved
           (+ kv_page_copy)              together, in every layer
  prefix   attn_paged_prefix             attention of one new token per request, the prefix that a group
                                         of requests shares computed once for all of them

`own` false: the plain forms, in elementary torch operations (32 bits; the scores of beams,
whose order is the answer, in 64).  `own` true: this package's calls.  Head counts and sizes
are those of the package's own shapes (4 KV heads of 128 with 8 query heads each; the decode
chain's 40 query and 4 KV heads of 128 and its 152064 output rows; depth 32768) or generic.
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
        # one request's four beams, the chain's vocabulary
        {"name": "beam 1 x 4 x 152064", "op": "beam", "requests": 1, "beams": 4, "vocab": 152064, "x": "fp32",
         "scale": 1.0, "ends": 1, "masked": False},
        # a step of 16 requests with four beams each, some tokens forbidden
        {"name": "beam 16 x 4 x 152064", "op": "beam", "requests": 16, "beams": 4, "vocab": 152064, "x": "fp32",
         "scale": 1.0, "ends": 1, "masked": True},
        # many beams of many requests over an odd vocabulary in bf16, no end token
        {"name": "beam 60 x 10 x 50021 bf16", "op": "beam", "requests": 60, "beams": 10, "vocab": 50021, "x": "bf16",
         "scale": 1.25, "ends": 0, "masked": False},
        # the survivors of four requests' beams, one layer
        {"name": "fork 4 x 4 of 1000", "op": "fork", "groups": 4, "beams": 4, "cached": 1000, "page": 16,
         "kv_heads": 4, "dim": 128, "cache": "fp16", "nhd": True, "layers": 1},
        # a server's beams at depth, four layers of large pages
        {"name": "fork 64 x 8 of 8192", "op": "fork", "groups": 64, "beams": 8, "cached": 8192, "page": 64,
         "kv_heads": 4, "dim": 128, "cache": "bf16", "nhd": False, "layers": 4},
        # after a fork: the pages of the beams that were dropped go back to the free list
        {"name": "free 64 rows of 8192", "op": "compact", "rows": 64, "cached": 8192, "page": 16, "kv_heads": 4,
         "dim": 128, "cache": "fp16", "nhd": True, "layers": 0, "moves": 0, "live": 0.7},
        # a pool with holes packed together, two layers
        {"name": "compact 40 rows of 2000", "op": "compact", "rows": 40, "cached": 2000, "page": 16, "kv_heads": 4,
         "dim": 128, "cache": "fp16", "nhd": True, "layers": 2, "moves": 4096, "live": 0.5},
        # a large pool of large pages, as many moves as there are
        {"name": "compact 300 rows of 8192", "op": "compact", "rows": 300, "cached": 8192, "page": 64, "kv_heads": 4,
         "dim": 128, "cache": "bf16", "nhd": False, "layers": 1, "moves": 20000, "live": 0.6},
        # one request's four beams over a prompt that ends inside a page
        {"name": "prefix 1 x 4 over 1000", "op": "prefix", "groups": 1, "per": 4, "prefix": 1000, "rest": 60,
         "kv_heads": 8, "group": 4, "dim": 64, "q": "fp16", "cache": "fp16", "page": 16, "nhd": True, "softcap": 0.0,
         "slopes": False},
        # sixteen prompts with four beams each at the chain's head counts
        {"name": "prefix 16 x 4 over 4096 bf16 g10", "op": "prefix", "groups": 16, "per": 4, "prefix": 4096,
         "rest": 300, "kv_heads": 4, "group": 10, "dim": 128, "q": "bf16", "cache": "bf16", "page": 64, "nhd": False,
         "softcap": 0.0, "slopes": False},
        # a system prompt of the configured depth in q8_0 pages, fp32 queries
        {"name": "prefix 1 x 33 over 32768 q8_0", "op": "prefix", "groups": 1, "per": 33, "prefix": 32768, "rest": 700,
         "kv_heads": 4, "group": 8, "dim": 128, "q": "fp32", "cache": "q8_0", "page": 32, "nhd": False, "softcap": 0.0,
         "slopes": False},
        # a large batch behind one system prompt
        {"name": "prefix 1 x 256 over 32768 bf16", "op": "prefix", "groups": 1, "per": 256, "prefix": 32768,
         "rest": 512, "kv_heads": 4, "group": 8, "dim": 128, "q": "bf16", "cache": "bf16", "page": 64, "nhd": True,
         "softcap": 0.0, "slopes": False},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["beam", "beam", "fork", "compact", "prefix", "prefix"])
    if op == "beam":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 10, 16])
        requests = _spread(rng, 1, max(1, 600 // beams))
        return {"op": op, "requests": requests, "beams": beams,
                "vocab": _spread(rng, 1000, min(260000, 30_000_000 // (requests * beams))),
                "x": rng.choice(["fp32", "fp16", "bf16"]), "scale": rng.choice([1.0, 1.25, 0.7]),
                "ends": rng.choice([0, 1, 1]), "masked": rng.random() < 0.4}
    kv_heads = rng.choice([1, 2, 4, 8])
    page, nhd, cache = rng.choice([8, 16, 32, 64, 128]), rng.random() < 0.5, rng.choice(["fp16", "bf16"])
    if op == "fork":
        dim = rng.choice([64, 128, 256])
        beams, groups = rng.choice([2, 3, 4, 8, 16]), _spread(rng, 1, 32)
        cached = _spread(rng, 10, 8192)
        rows = groups * (cached + 2 * beams * page)  # positions in the pool
        most = 64 * 16384 * 4 * 128 * 4 // (rows * kv_heads * dim)
        return {"op": op, "groups": groups, "beams": beams, "cached": cached, "page": page, "kv_heads": kv_heads,
                "dim": dim, "cache": cache, "nhd": nhd, "layers": max(1, min(4, most))}
    if op == "compact":
        dim = rng.choice([64, 128, 256])
        rows = _spread(rng, 1, 300)
        cached = _spread(rng, 10, max(10, 300 * 8192 * 4 * 128 // (rows * kv_heads * dim)) if rows > 30 else 30000)
        moves = rng.choice([0, _spread(rng, 1, 20000), 20000])
        layers = min(2, max(1, 300 * 8192 * 4 * 128 // (rows * cached * kv_heads * dim))) if moves else 0
        return {"op": op, "rows": rows, "cached": cached, "page": page, "kv_heads": kv_heads, "dim": dim,
                "cache": cache, "nhd": nhd, "layers": layers, "moves": moves, "live": rng.choice([0.3, 0.6, 0.9])}
    dim = rng.choice([64, 128, 128])
    q, cache = rng.choice([("fp32", "fp16"), ("fp32", "q8_0"), ("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "q8_0"),
                           ("fp32", "bf16")])
    groups, group = _spread(rng, 1, 40), rng.choice([1, 2, 3, 4, 7, 8, 10, 16])
    per = _spread(rng, 1, max(1, 256 // groups))
    limit = 256 * 32768 * 8 * 4 * 128 // (groups * per * group * kv_heads * dim)
    deep = min(32768, limit // (3 if q == "fp32" else 1), 4 * 32768 * 4 * 128 // (groups * kv_heads * dim))
    return {"op": op, "groups": groups, "per": per, "prefix": _spread(rng, 1, max(2, deep)),
            "rest": _spread(rng, 1, max(2, min(2000, 256 * 512 * 4 * 128 // (groups * per * kv_heads * dim)))),
            "kv_heads": kv_heads, "group": group, "dim": dim, "q": q, "cache": cache, "page": page, "nhd": nhd,
            "softcap": rng.choice([0.0, 0.0, 30.0]), "slopes": rng.random() < 0.2}


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(1_000_003 * seed + 29)


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int64)


def _pages(n, page):
    return (n + page - 1) // page


def _i32(*shape, fill=None):
    if fill is None:
        return torch.empty(*shape, dtype=torch.int32, device="cuda")
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    return {"case": case, **{"beam": _prepare_beam, "fork": _prepare_fork, "compact": _prepare_compact,
                             "prefix": _prepare_prefix}[case["op"]](case, g)}


def _prepare_beam(c, g):
    n, k, v = c["requests"], c["beams"], c["vocab"]
    # the beams of a request have a prompt in common: their rows resemble each other
    x = torch.randn(n, 1, v, generator=g, device="cuda").mul(2.0) + torch.randn(n, k, v, generator=g, device="cuda").mul_(1.5)
    if c["masked"]:
        x.masked_fill_(torch.rand(n, k, v, generator=g, device="cuda") < 0.01, -math.inf)
    if c["ends"]:  # the end token is likely in a quarter of the rows
        x[..., 2] = torch.where(torch.rand(n, k, generator=g, device="cuda") < 0.25, 9.0, -3.0) + \
            torch.randn(n, k, generator=g, device="cuda")
    score = torch.rand(n, k, generator=g, device="cuda").mul_(4).cumsum(1).neg_() - 10
    s = {"logits": x.view(n * k, v).to(_T[c["x"]]), "scores": score.contiguous(), "ends": [2] * c["ends"]}
    if own:
        s["out"] = _lib().beam_select_out(n, k, device="cuda")
        s["ws"] = torch.zeros(max(16, _lib().beam_select_workspace_bytes(n, k, v, c["ends"])), dtype=torch.uint8,
                              device="cuda")
    return s


def _layer(c, pages, g):
    """k and v of one layer's cache with `pages` pages of normal values, in the case's layout."""
    h, d, p = c["kv_heads"], c["dim"], c["page"]
    shape = (pages, p, h, d) if c["nhd"] else (pages, h, p, d)
    return [torch.randn(shape, generator=g, device="cuda", dtype=_T[c["cache"]]) for _ in range(2)]


def _handles(c, layers):
    return [_lib().PagedKV(k, v, layout="nhd" if c["nhd"] else "hnd") for k, v in layers] if own else None


def _copies(n, parts=True):
    return _lib().PageCopies(_i32(n), _i32(n), _i32(n) if parts else None, _i32(1)) if own else None


def _prepare_fork(c, g):
    groups, beams, page = c["groups"], c["beams"], c["page"]
    n = groups * beams
    # each group's beams share the pages of a prompt and have two pages each of their own, the last of them partly
    # filled (or, for one length in `page`, full)
    prompt = _ints(g, max(1, c["cached"] // 2), c["cached"], groups) // page
    width = c["cached"] // page + 3
    own_tokens = _ints(g, page + 1, 2 * page, groups)
    lens = ((prompt * page + own_tokens)[:, None].expand(groups, beams)).reshape(-1)
    j = torch.arange(width, device="cuda")[None, :]
    shared = prompt.repeat_interleave(beams)[:, None]
    total = int(prompt.sum()) + 2 * n
    pool = groups * (c["cached"] // page) + 3 * n + 7
    ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    first = (torch.cumsum(prompt, 0) - prompt).repeat_interleave(beams)[:, None]
    row = torch.arange(n, device="cuda")[:, None]
    at = torch.where(j < shared, first + j, int(prompt.sum()) + 2 * row + (j - shared).clamp(0, 1))
    table = torch.where(j < shared + 2, ids[at], -1).to(torch.int32).contiguous()
    # the children of a step: a few parents have several, some have none
    parent = _ints(g, 0, beams - 1, n).view(groups, beams).square().div(beams, rounding_mode="floor")
    parent = (parent + beams * torch.arange(groups, device="cuda")[:, None]).reshape(-1).to(torch.int32)
    layers = [_layer(c, pool, g) for _ in range(c["layers"])]
    s = {"parent": parent, "lens": lens.to(torch.int32), "table": table, "free": ids[total:].contiguous(),
         "head": _i32(1, fill=0), "layers": layers, "handles": _handles(c, layers), "pages": pool}
    if own:
        s["out"] = _lib().KvFork(_i32(n, width, fill=-1), _i32(n), _i32(1), _copies(n))
    else:
        s["blank"] = _i32(n, width, fill=-1)
    return s


def _prepare_compact(c, g):
    n, page = c["rows"], c["page"]
    low = max(1, c["cached"] // 2)
    lens = _ints(g, low, c["cached"], n)
    lens[n - n // 2:] = low + c["cached"] - lens[: n // 2]  # pairs of the same sum: a pool of fixed size
    need = _pages(lens, page)
    width = _pages(c["cached"], page) + 1
    total = int(need.sum())
    most = n // 2 * ((low + c["cached"]) // page + 2) + n % 2 * _pages(c["cached"], page)
    pool = int(most / c["live"]) + most // 50 + 5
    ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = _i32(n, width, fill=-1)
    table[torch.arange(width, device="cuda")[None, :] < need[:, None]] = ids[:total]
    held = torch.zeros(pool, dtype=torch.uint8, device="cuda")
    held[ids[total:total + pool // 100].long()] = 1  # a few pages that a prefix store holds
    layers = [_layer(c, pool, g) for _ in range(c["layers"])]
    s = {"lens": lens.to(torch.int32), "table": table, "held": held, "pages": pool, "layers": layers,
         "handles": _handles(c, layers), "moves": min(c["moves"], pool)}
    if own:
        s["out"] = _lib().KvCompact(_i32(n, width, fill=-1) if s["moves"] else table, _i32(pool, fill=-1), _i32(1),
                                    _copies(s["moves"], parts=False))
        s["ws"] = torch.zeros(_lib().kv_page_compact_workspace_bytes(pool), dtype=torch.uint8, device="cuda")
    return s


def _prepare_prefix(c, g):
    groups, per, h, d, page = c["groups"], c["per"], c["kv_heads"], c["dim"], c["page"]
    n, heads = groups * per, h * c["group"]
    prefix = _ints(g, max(1, c["prefix"] // 2), c["prefix"], groups)
    prefix[0] = c["prefix"]
    rest = _ints(g, 1, c["rest"], n)
    plen = prefix.repeat_interleave(per)
    lens = plen + rest
    if n >= 8:
        lens[n // 2] = 0  # an unused row of a padded batch
    width = _pages(c["prefix"] + c["rest"], page)
    j = torch.arange(width, device="cuda")[None, :]
    whole = (prefix // page)  # a group's whole pages; the one in which the prefix ends is each request's own
    mine = (_pages(plen + rest, page) - whole.repeat_interleave(per))
    total = int(whole.sum()) + int(mine.sum())
    ids = torch.randperm(total + 3, generator=g, device="cuda").to(torch.int32)
    first = (torch.cumsum(whole, 0) - whole).repeat_interleave(per)[:, None]
    first_mine = (int(whole.sum()) + torch.cumsum(mine, 0) - mine)[:, None]
    w = whole.repeat_interleave(per)[:, None]
    at = torch.where(j < w, first + j, (first_mine + j - w).clamp(max=total))
    table = torch.where(j < w + mine[:, None], ids[at], -1).to(torch.int32).contiguous()
    shape = (total + 3, page, h) if c["nhd"] else (total + 3, h, page)
    if c["cache"] == "q8_0":
        kv = [torch.randint(-127, 128, (*shape, d), generator=g, device="cuda", dtype=torch.int8) for _ in range(2)]
        kv += [((torch.rand(*shape, d // 32, generator=g, device="cuda") + 1.5) / 127).half() for _ in range(2)]
    else:
        kv = [torch.randn(*shape, d, generator=g, device="cuda", dtype=_T[c["cache"]]) for _ in range(2)] + [None, None]
    _same_first_part(c, kv, table, prefix, per)
    s = {"q": torch.randn(n, heads, d, generator=g, device="cuda").to(_T[c["q"]]), "kv": kv, "table": table,
         "lens": lens.to(torch.int32), "prefix": prefix.to(torch.int32), "scale": 1 / math.sqrt(d), "slopes": None,
         "groups": (torch.arange(groups + 1, device="cuda") * per).to(torch.int32),
         "out": torch.empty(n, heads, d, dtype=_T[c["q"]], device="cuda"),
         "lse": torch.empty(n, heads, dtype=torch.float32, device="cuda")}
    if c["slopes"]:
        s["slopes"] = 2.0 ** (-8 * torch.arange(1, heads + 1, device="cuda") / heads)
    if own:
        s["handle"] = _lib().PagedKV(*kv, layout="nhd" if c["nhd"] else "hnd")
        s["ws"] = torch.zeros(_lib().attn_paged_prefix_workspace_bytes(n, groups, heads, h, d), dtype=torch.uint8,
                              device="cuda")
    return s


def _same_first_part(c, kv, table, prefix, per):
    """The page in which a prefix ends is a copy in each request's own page: its part of the prefix is
    that of the group's first request."""
    page, groups = c["page"], c["groups"]
    last = (prefix // page).clamp(max=table.shape[1] - 1)
    pages = table.view(groups, per, -1).gather(2, last[:, None, None].expand(groups, per, 1))[..., 0].clamp(min=0).long()
    part = torch.arange(page, device="cuda")[None, :] < (prefix % page)[:, None]  # [groups][page]
    mask = part[:, None, :, None, None] if c["nhd"] else part[:, None, None, :, None]
    for x in kv:
        if x is not None:
            rows = x[pages]  # [groups][per][page ..]
            x[pages.view(-1)] = torch.where(mask, rows[:, :1], rows).flatten(0, 1)


# -------------------------------------------------------------- one pass --

def run(state):
    return {"beam": _beam, "fork": _fork, "compact": _compact, "prefix": _prefix}[state["case"]["op"]](state)


def _beam(s):
    c = s["case"]
    n, k, v = c["requests"], c["beams"], c["vocab"]
    if own:
        r = _lib().beam_select(s["logits"], s["scores"], s["ends"], scale=c["scale"], out=s["out"], ws=s["ws"])
        return {"parent": r.parent, "token": r.token, "score": r.score, "end_parent": r.end_parent,
                "end_token": r.end_token, "end_score": r.end_score}
    y = s["logits"].double() * c["scale"]
    m = y.amax(-1, keepdim=True)
    logprob = y - (m + torch.log(torch.exp(y - m).sum(-1, keepdim=True)))
    total = (s["scores"].double().view(n * k, 1) + logprob).view(n, k * v)
    want = k * (1 + c["ends"])
    best, at = torch.sort(total, dim=1, descending=True, stable=True)  # equal ones: the lower index
    best, at = best[:, :want], at[:, :want]
    token, parent = at % v, at // v + k * torch.arange(n, device=at.device)[:, None]
    ended = token == 2 if c["ends"] else torch.zeros_like(token, dtype=torch.bool)
    there = best > -math.inf
    alive = there & ~ended
    rank = torch.arange(want, device=at.device)[None, :]
    got = {}
    for name, which in (("", alive & (alive.cumsum(1) <= k)), ("end_", there & ended & (rank < k))):
        place = torch.where(which, which.cumsum(1) - 1, k)  # the others fall into a place that is cut off
        for what, value, none in (("parent", parent.int(), -1), ("token", token.int(), -1),
                                  ("score", best.float(), -math.inf)):
            room = torch.full((n, k + 1), none, dtype=value.dtype, device=at.device)
            got[name + what] = room.scatter_(1, place, value)[:, :k]
    return got


def _copied(layers, src, dst, which, fill, c):
    """Pages src to dst where `which`, their first `fill` positions."""
    last = layers[0][0].shape[0] if layers else 0
    part = torch.arange(c["page"], device=src.device)[None, :] < fill[:, None]
    part = part[:, :, None, None] if c["nhd"] else part[:, None, :, None]
    for k, v in layers:
        for x in (k, v):
            # entries that copy nothing write a page's own values to it: to the page that they would read
            to = torch.where(which, dst, src).clamp(0, last - 1)
            x[to] = torch.where(part & which[:, None, None, None], x[src.clamp(0, last - 1)], x[to])


def _fork(s):
    c = s["case"]
    page = c["page"]
    if own:
        r = _lib().kv_page_fork(s["parent"], s["lens"], s["free"], s["head"], s["table"], page, out=s["out"])
        _lib().kv_page_copy(r.copies, s["handles"])
        return {"table": r.table, "lens": r.seq_len, "head": r.head, "count": r.copies.count,
                "layers": s["layers"]}
    parent, n = s["parent"].long(), s["parent"].numel()
    lens = s["lens"].long()[parent]
    need = _pages(lens, page)
    row = torch.arange(n, device=parent.device)
    lowest = torch.full_like(parent, n).scatter_reduce(0, parent, row, "amin")
    copy = (lens % page != 0) & (lowest[parent] != row)
    k = copy.cumsum(0)
    fresh = s["free"].long()[(s["head"].long() + k - 1).clamp(min=0)]
    j = torch.arange(s["table"].shape[1], device=parent.device)[None, :]
    old = s["table"].long()[parent]
    table = torch.where(copy[:, None] & (j == need[:, None] - 1), fresh[:, None], old)
    src = old.gather(1, (need - 1).clamp(min=0)[:, None])[:, 0]
    _copied(s["layers"], src, fresh, copy, lens % page, c)
    return {"table": torch.where(j < need[:, None], table, s["blank"].long()).int(), "lens": lens.int(),
            "head": (s["head"] + k[-1]).int(), "count": k[-1:].int(), "layers": s["layers"]}


def _compact(s):
    c, pool, moves = s["case"], s["pages"], s["moves"]
    if own:
        r = _lib().kv_page_compact(s["lens"], s["table"], c["page"], pool, held=s["held"], max_moves=moves, out=s["out"],
                                   ws=s["ws"])
        if moves:
            _lib().kv_page_copy(r.copies, s["handles"])
        return {"table": r.table, "free": r.free_pages, "head": r.head, "count": r.copies.count, "layers": s["layers"]}
    need = _pages(s["lens"].long(), c["page"])
    j = torch.arange(s["table"].shape[1], device=need.device)[None, :]
    listed_ = j < need[:, None]
    at = torch.where(listed_, s["table"].long(), pool)
    marks = torch.zeros(pool + 1, dtype=torch.bool, device=need.device)
    marks[at.view(-1)] = True
    mine, held = marks[:pool], s["held"] != 0
    live = mine | held
    ids = torch.arange(pool, device=need.device)
    many = live.sum()
    movable, hole = live & ~held & (ids >= many), ~live & (ids < many)
    out_rank, in_rank = movable.cumsum(0) - 1, hole.cumsum(0) - 1
    count = torch.minimum(movable.sum(), hole.sum()).clamp(max=moves)
    moved, filled = movable & (out_rank < count), hole & (in_rank < count)
    dst = torch.zeros(pool + 1, dtype=torch.int64, device=need.device)
    dst[torch.where(filled, in_rank, pool)] = ids  # the place of the others is not read
    to = torch.where(moved, dst[out_rank.clamp(min=0)], ids)
    table = torch.where(listed_, to[at.clamp(max=pool - 1)], -1)
    if moves:
        src = torch.zeros(pool + 1, dtype=torch.int64, device=need.device)
        src[torch.where(moved, out_rank, pool)] = ids
        # a move of every rank up to the most that there can be; those past the count move nothing
        rank = torch.arange(min(moves, pool), device=need.device)
        which = rank < count
        own_page = torch.where(which, src[:rank.numel()], rank)
        _moved(s["layers"], own_page, torch.where(which, dst[:rank.numel()], rank), which)
    empty = ~((live & ~moved) | filled)
    free_at = torch.where(empty, empty.cumsum(0) - 1 + pool - empty.sum(), pool)
    free = torch.full((pool + 1,), -1, dtype=torch.int64, device=need.device)
    free[free_at] = ids
    return {"table": table.int() if moves else s["table"], "free": free[:pool].int(),
            "head": (pool - empty.sum()).int().view(1), "count": count.int().view(1), "layers": s["layers"]}


def _moved(layers, src, dst, which):
    for k, v in layers:
        for x in (k, v):
            pages = x[src]
            keep = torch.where(which, dst, x.shape[0])
            room = torch.cat([x, x[:1]])  # a place for the entries that move nothing
            room[keep] = pages
            x.copy_(room[:-1])


def _values(codes, scales):
    """What q8_0 codes stand for, in fp16."""
    return (codes.float().unflatten(-1, (-1, 32)) * scales.float()[..., None]).flatten(-2).half()


def _gathered(s, i, pages, first, count):
    """K (0) or V (1) at `count` positions from first[r] on of the block table rows `pages`, in fp32:
    [rows][kv heads][positions][dim]."""
    c, kv = s["case"], s["kv"]
    p = first[:, None] + torch.arange(count, device=first.device)[None, :]
    page = pages.long().gather(1, (p // c["page"]).clamp(max=pages.shape[1] - 1)).clamp(min=0)
    off = p % c["page"]
    x = kv[i][page, off] if c["nhd"] else kv[i][page, :, off]
    if c["cache"] == "q8_0":
        x = _values(x, kv[2 + i][page, off] if c["nhd"] else kv[2 + i][page, :, off])
    return x.transpose(1, 2).float()


def _prefix(s):
    c = s["case"]
    if own:
        _lib().attn_paged_prefix(s["q"], s["handle"], s["table"], s["lens"], s["groups"], s["prefix"], scale=s["scale"],
                                 softcap=c["softcap"], slopes=s["slopes"], out=s["out"], lse=s["lse"], ws=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    groups, per, h, group, d = c["groups"], c["per"], c["kv_heads"], c["group"], c["dim"]
    n, long, rest = groups * per, c["prefix"], c["rest"]
    lens, prefix = s["lens"].long(), s["prefix"].long()
    plen = prefix.repeat_interleave(per)
    q = s["q"].float()

    def scores(x, p, r):  # of [n][h][group][positions] at positions p for the lengths r
        x = x * s["scale"]
        if c["softcap"]:
            x = c["softcap"] * torch.tanh(x / c["softcap"])
        if c["slopes"]:
            x = x - s["slopes"].float().reshape(1, h, group, 1) * (r[:, None] - 1 - p).reshape(n, 1, 1, -1)
        return x

    zero = torch.zeros_like(prefix)
    rows = s["table"].reshape(groups, per, -1)[:, 0]
    qg = q.reshape(groups, per, h, group, d).permute(0, 2, 1, 3, 4).reshape(groups, h, per * group, d)
    xs = (qg @ _gathered(s, 0, rows, zero, long).transpose(2, 3)).reshape(groups, h, per, group, long)
    p = torch.arange(long, device=q.device)[None, :]
    xs = scores(xs.permute(0, 2, 1, 3, 4).reshape(n, h, group, long), p, lens)
    seen = (p < plen[:, None]) & (p < lens[:, None])
    xs = torch.where(seen[:, None, None, :], xs, -math.inf)
    xo = q.reshape(n, h, group, d) @ _gathered(s, 0, s["table"], plen, rest).transpose(2, 3)
    p = plen[:, None] + torch.arange(rest, device=q.device)[None, :]
    xo = torch.where((p < lens[:, None])[:, None, None, :], scores(xo, p, lens), -math.inf)
    m = torch.maximum(xs.amax(-1, keepdim=True), xo.amax(-1, keepdim=True))
    ref = torch.where(m == -math.inf, 0.0, m)
    ws, wo = torch.exp(xs - ref), torch.exp(xo - ref)
    total = ws.sum(-1, keepdim=True) + wo.sum(-1, keepdim=True)
    wg = ws.reshape(groups, per, h, group, long).permute(0, 2, 1, 3, 4).reshape(groups, h, per * group, long)
    part = (wg @ _gathered(s, 1, rows, zero, long)).reshape(groups, h, per, group, d).permute(0, 2, 1, 3, 4)
    out = part.reshape(n, h, group, d) + wo @ _gathered(s, 1, s["table"], plen, rest)
    out = out / torch.where(total == 0, 1.0, total)
    return {"out": out.reshape(n, h * group, d).to(s["q"].dtype), "lse": (m + torch.log(total)).reshape(n, h * group)}


# ------------------------------------------------------------------- work --

def work(case):
    c = case
    if c["op"] == "beam":
        rows = c["requests"] * c["beams"]
        return {"bytes": rows * (c["vocab"] * _BYTES[c["x"]] + 28.0), "flops": 5.0 * rows * c["vocab"]}
    row = 2.0 * c["kv_heads"] * c["dim"] * _BYTES[c["cache"]]  # K and V of a position
    if c["op"] == "fork":
        n = c["groups"] * c["beams"]
        entries = n * (0.75 * c["cached"] / c["page"] + 2)
        # table rows in and out; about half of the rows are other rows' children and copy half a page
        return {"bytes": 8.0 * entries + 24.0 * n + c["layers"] * 0.5 * n * 0.5 * c["page"] * 2 * row, "flops": 0.0}
    if c["op"] == "compact":
        entries = 0.75 * c["rows"] * c["cached"] / c["page"]
        pool = entries / c["live"]
        moved = min(c["moves"], entries * (1 - c["live"]))
        return {"bytes": (8.0 if c["moves"] else 4.0) * entries + 5.0 * pool - 4.0 * entries
                + c["layers"] * moved * c["page"] * 2 * row, "flops": 0.0}
    n, heads = c["groups"] * c["per"], c["kv_heads"] * c["group"]
    prefix = c["prefix"] + max(0, c["groups"] - 1) * 0.75 * c["prefix"]  # the first is the longest, the others even
    rest = 0.5 * n * c["rest"]
    return {"bytes": (prefix + rest) * row + n * heads * (2 * c["dim"] * _BYTES[c["q"]] + 4),
            "flops": 4.0 * heads * c["dim"] * (c["per"] * prefix + rest)}


# ------------------------------------------------------- 64-bit definition --

def exact(case, seed):
    """What run() returns, computed in 64 bits a request at a time."""
    if case["op"] in ("fork", "compact"):
        return None  # whole numbers, and values that are moved
    s = prepare(case, seed)
    return (_exact_beam if case["op"] == "beam" else _exact_prefix)(case, s)


def _exact_beam(c, s):
    n, k, v = c["requests"], c["beams"], c["vocab"]
    want = k * (1 + c["ends"])
    score = torch.full((n, k), -math.inf, dtype=torch.float64, device="cuda")
    ended = score.clone()
    for r in range(n):
        lp = torch.log_softmax(s["logits"][r * k:(r + 1) * k].double() * c["scale"], -1)
        all_ = s["scores"][r].double()[:, None] + lp
        end = all_[:, 2].clone()
        if c["ends"]:
            all_[:, 2] = -math.inf
        alive = all_.flatten().topk(min(k, all_.numel())).values
        score[r, :alive.numel()] = alive
        if c["ends"]:
            both = torch.cat([all_.flatten().topk(min(want, all_.numel())).values, end])
            order = both.argsort(descending=True)[:k]
            done = both[order[order >= both.numel() - k]]
            ended[r, :done.numel()] = done
    return {"parent": None, "token": None, "score": score, "end_parent": None, "end_token": None, "end_score": ended}


def _exact_prefix(c, s):
    h, group, d, per = c["kv_heads"], c["group"], c["dim"], c["per"]
    n = c["groups"] * per
    out = torch.zeros(n, h * group, d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, h * group), -math.inf, dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    for r in range(n):
        if lens[r] == 0:
            continue
        p = torch.arange(lens[r], device="cuda")
        page, off = s["table"][r].long()[p // c["page"]], p % c["page"]
        got = []
        for i in range(2):
            x = s["kv"][i][page, off] if c["nhd"] else s["kv"][i][page, :, off]  # [positions][heads][dim]
            if c["cache"] == "q8_0":
                f = s["kv"][2 + i][page, off] if c["nhd"] else s["kv"][2 + i][page, :, off]
                x = (x.double() * f.double().repeat_interleave(32, -1)).half()  # a cached value is binary16
            got.append(x.double().transpose(0, 1))
        q = s["q"][r].double().view(h, group, d)
        x = q @ got[0].transpose(1, 2) * s["scale"]
        if c["softcap"]:
            x = c["softcap"] * torch.tanh(x / c["softcap"])
        if c["slopes"]:
            x = x + s["slopes"].double().view(h, group, 1) * (p - (lens[r] - 1)).double()
        lse[r] = torch.logsumexp(x, -1).reshape(-1)
        out[r] = (torch.softmax(x, -1) @ got[1]).reshape(-1, d)
    return {"out": out, "lse": lse}
