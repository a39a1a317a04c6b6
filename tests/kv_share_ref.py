"""Plain forms of the operators for rows that share pages, for the tests: loops over the
definitions in wsw.h, which share nothing with the library."""
import math

import numpy as np


def pages(n, page):
    return -(-n // page)


def fork(parent, seq, free, head, table, page, rows_out=None):
    """(table, lens, head, [(src, dst, fill)], err) of wsw_kv_page_fork; entries that the call leaves
    alone come from rows_out (the new table's contents before)."""
    width = table.shape[1]
    out = (np.full((len(parent), width), -7) if rows_out is None else rows_out).copy()
    fits = [n >= 0 and pages(n, page) <= width for n in map(int, seq)]
    reach = max([pages(int(n), page) for n, f in zip(seq, fits) if f], default=0)
    lens, copies, err, seen = [], [], 0, set()
    avail = len(free) - head if 0 <= head <= len(free) else 0
    for i, p in enumerate(map(int, parent)):
        if p < -1 or p >= len(seq):
            err |= 1
            p = -1
        if p >= 0 and not fits[p]:
            err |= 2
            p = -1
        n = int(seq[p]) if p >= 0 else 0
        row = list(table[p, :pages(n, page)]) if p >= 0 else []
        if n % page:
            if p in seen:
                if len(copies) < avail:
                    fresh = int(free[head + len(copies)])
                    copies.append((int(row[-1]), fresh, n % page))
                    row[-1] = fresh
                else:
                    err |= 8
                    n, row = 0, []
            seen.add(p)
        out[i, :reach] = row + [-1] * (reach - len(row))
        lens.append(n)
    return out, np.array(lens, np.int64), head + len(copies), copies, err


def compact(seq, table, page, num_pages, held=None, max_moves=0):
    """(table, free pages, head, [(src, dst)], err) of wsw_kv_page_compact."""
    out, err = table.copy(), 0
    listed = set()
    used = []
    for r, n in enumerate(map(int, seq)):
        if n < 0 or pages(n, page) > table.shape[1]:
            err |= 2
            continue
        for j in range(pages(n, page)):
            e = int(table[r, j])
            if 0 <= e < num_pages:
                listed.add(e)
                used.append((r, j))
            else:
                err |= 1
    stay = set() if held is None else {p for p in range(num_pages) if held[p]}
    live = listed | stay
    many = len(live)
    movable = [p for p in sorted(listed - stay) if p >= many]
    holes = [p for p in range(many) if p not in live]
    moves = list(zip(movable, holes))[:max_moves]
    to = dict(moves)
    for r, j in used:
        out[r, j] = to.get(int(table[r, j]), int(table[r, j]))
    live = (live - set(to)) | set(to.values())
    return out, [p for p in range(num_pages) if p not in live], many, moves, err


def attend(q, k, v, scale, softcap=0.0, slopes=None, distance=None):
    """One request in float64: q [heads][dim], k and v [positions][kv heads][dim].  Returns out, lse and the
    weighted magnitudes sum w |v| / sum w."""
    heads, kvh = q.shape[0], k.shape[1]
    g = heads // kvh
    qg = q.reshape(kvh, g, -1)
    x = np.einsum("hgd,phd->hgp", qg, k) * scale
    if softcap:
        x = softcap * np.tanh(x / softcap)
    if slopes is not None:
        x = x - slopes.reshape(kvh, g, 1) * distance
    m = x.max(-1, keepdims=True)
    w = np.exp(x - m)
    t = w.sum(-1, keepdims=True)
    out = np.einsum("hgp,phd->hgd", w, v) / t
    mag = np.einsum("hgp,phd->hgd", w, np.abs(v)) / t
    return out.reshape(heads, -1), (m + np.log(t)).reshape(heads), mag.reshape(heads, -1)


def beam(logits, scores, ends, scale=1.0):
    """One request in float64: logits [beams][vocab], scores [beams].  Returns ([(beam, token, score)] of the next
    beams, the same of the ended candidates, the scores in order up to the first that was not taken)."""
    beams, vocab = logits.shape
    total = np.full((beams, vocab), -np.inf)
    for b in range(beams):
        x = logits[b].astype(np.float64) * scale
        m = x.max()
        if not np.isfinite(m) or np.isnan(x).any() or not scores[b] < np.inf:
            continue
        # x - m first: it stays exact where m + ln S itself is huge (a row at the type's lowest value)
        total[b] = scores[b] + ((x - m) - math.log(np.exp(x - m).sum()))
    flat = total.ravel()
    order = np.lexsort((np.arange(flat.size), -flat))
    nxt, ended = [], []
    for rank, i in enumerate(order):
        if flat[i] == -np.inf or len(nxt) == beams:
            break
        c = (int(i) // vocab, int(i) % vocab, float(flat[i]))
        if c[1] in ends:
            if rank < beams:
                ended.append(c)
        else:
            nxt.append(c)
    return nxt, ended, flat[order[: rank + 1]]
