"""Plain 64-bit forms of the operators around the paged KV cache, for the tests.  They are
loops and numpy over the definitions in wsw.h and share nothing with the library."""
import math

import numpy as np


def page_plan(seq, new, free, head, table, page, tokens):
    """(table, positions, slots, cu, lens, head, err) of wsw_kv_page_plan."""
    table = table.copy()
    width = table.shape[1]
    n = len(seq)
    pos = np.full(tokens, -1, np.int64)
    slot = np.full(tokens, -1, np.int64)
    cu = np.zeros(n + 1, np.int64)
    lens = np.array(seq, np.int64)
    err = at = taken = granted = 0
    avail = len(free) - head if 0 <= head <= len(free) else 0
    for r in range(n):
        s, k = int(seq[r]), int(new[r])
        cu[r] = min(at, tokens)
        if s < 0 or k < 0:
            err |= 1
            continue
        begin, at = at, at + k
        want, have = -(-(s + k) // page), -(-s // page)
        if want > width or s + k > 0x7fffffff:
            err |= 2
            continue
        if at > tokens:
            err |= 4
            continue
        need = want - have
        first, taken = taken, taken + need
        if need and taken > avail:
            err |= 8
            continue
        granted = max(granted, taken) if need else granted
        table[r, have:want] = free[head + first: head + first + need]
        lens[r] = s + k
        for i in range(k):
            p = s + i
            pos[begin + i] = p
            pg = int(table[r, p // page])
            slot[begin + i] = pg * page + p % page if pg >= 0 else -1
    cu[n] = min(at, tokens)
    return table, pos, slot, cu, lens, head + granted, err


def rope_freqs(rot, theta=10000.0, scaling=None, factor=1.0, original=0):
    """(radians per position of each pair, factor on cos and sin)."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = theta ** (-2 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "by_parts":
        turns = original * f / (2 * math.pi)
        keep = np.clip((turns - 1) / 31, 0, 1)
        return keep * f + (1 - keep) * f / factor, 0.1 * math.log(factor) + 1
    return f, 1.0


def rotate(x, positions, f, m, interleaved):
    """x [tokens][heads][dim] in float64."""
    r = 2 * len(f)
    y = x.copy()
    ang = positions.astype(np.float64)[:, None] * f
    c, s = m * np.cos(ang)[:, None], m * np.sin(ang)[:, None]
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., : r // 2], x[..., r // 2: r]
        y[..., : r // 2], y[..., r // 2: r] = a * c - b * s, b * c + a * s
    return y


def attend(q, k, v, scale, softcap=0.0, slopes=None, distance=None):
    """One request: q [heads][dim], k and v [positions][kv heads][dim], in float64.  Returns
    out, lse, the weighted magnitudes sum w |v| / sum w, and max_p scale sum |q k|."""
    heads, kvh = q.shape[0], k.shape[1]
    g = heads // kvh
    qg = q.reshape(kvh, g, -1)
    x = np.einsum("hgd,phd->hgp", qg, k) * scale
    terms = float((np.einsum("hgd,phd->hgp", np.abs(qg), np.abs(k)) * abs(scale)).max())
    if softcap:
        x = softcap * np.tanh(x / softcap)
    if slopes is not None:
        x = x - slopes.reshape(kvh, g, 1) * distance
    m = x.max(-1, keepdims=True)
    w = np.exp(x - m)
    t = w.sum(-1, keepdims=True)
    out = np.einsum("hgp,phd->hgd", w, v) / t
    mag = np.einsum("hgp,phd->hgd", w, np.abs(v)) / t
    return out.reshape(heads, -1), (m + np.log(t)).reshape(heads), mag.reshape(heads, -1), terms


def logprobs(x, token, scale, top):
    """One row in float64: (logprob, rank, lse, entropy, top ids, top logprobs, ln S), with
    S = sum exp(y - max y): the probabilities come from y - max y, which stays exact where
    lse itself is huge (a row at the type's lowest value)."""
    y = x * scale
    m = y.max()
    order = np.lexsort((np.arange(len(x)), -x))[:top]
    rank = int((x > x[token]).sum() + (x[:token] == x[token]).sum())
    if m == -np.inf:
        return -np.inf, rank, -np.inf, 0.0, order, np.full(top, -np.inf), 0.0
    ln_s = math.log(np.exp(y - m).sum())
    lp = (y - m) - ln_s
    p = np.exp(lp)
    ent = -(p[p > 0] * lp[p > 0]).sum()
    return lp[token], rank, m + ln_s, ent, order, lp[order], ln_s
