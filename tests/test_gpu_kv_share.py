"""Forking, copying and compacting pages on the GPU against the plain loops: whole numbers and
moved values, equal everywhere."""
import numpy as np
import pytest
import torch

import kv_share_ref as ref
from helpers import need_gpu

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _rows(g, n, cached, page, shared=0):
    """Lengths and a table of n rows over distinct pages (the first `shared` columns in common)."""
    seq = g.integers(0, cached + 1, n)
    width = max(1, -(-cached // page) + 1)
    ids = g.permutation(n * width + 20)
    table = ids[: n * width].reshape(n, width).copy()
    if shared:
        table[:, :shared] = table[0, :shared]
    return seq, table, ids[n * width:]


def _fork(wsw, parent, seq, free, head, table, page, in_place=False, opts=None):
    before = None if not in_place else np.vstack([table, np.full((max(0, len(parent) - len(seq)), table.shape[1]), 3)])
    want = ref.fork(parent, seq, free, head, table, page,
                    before[:len(parent)] if in_place else np.full((len(parent), table.shape[1]), 55))
    n = len(parent)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    copies = wsw.PageCopies(*[_i32(np.full(n, 77)) for _ in range(3)], _i32([77]))
    if in_place:
        room = _i32(before)
        lens = _i32(np.concatenate([seq, np.zeros(max(0, n - len(seq)), int)]))
        head_d = _i32([head])
        out = wsw.KvFork(room[:n], lens[:n], head_d, copies)
        r = wsw.kv_page_fork(_i32(parent), lens[:len(seq)], _i32(free), head_d, room[:len(seq)], page, out=out, err_flag=err,
                             opts=opts)
        assert np.array_equal(room[n:].cpu().numpy(), before[n:])
    else:
        out = wsw.KvFork(_i32(np.full((n, table.shape[1]), 55)), _i32(np.full(n, 5)), _i32([5]), copies)
        table_d = _i32(table)
        r = wsw.kv_page_fork(_i32(parent), _i32(seq), _i32(free), _i32([head]), table_d, page, out=out, err_flag=err,
                             opts=opts)
        assert np.array_equal(table_d.cpu().numpy(), table)
    k = len(want[3])
    got = [t.cpu().numpy() for t in (r.copies.src, r.copies.dst, r.copies.fill)]
    assert np.array_equal(r.table.cpu().numpy(), want[0])
    assert r.seq_len.tolist() == want[1].tolist() and r.head.tolist() == [want[2]] and r.copies.count.tolist() == [k]
    assert [tuple(int(x[i]) for x in got) for i in range(k)] == want[3]
    assert all((x[k:] == 77).all() for x in got)
    assert int(err) == want[4]
    return want


@pytest.mark.parametrize("children,rows,cached,page", [
    (1, 1, 0, 16), (1, 1, 17, 16), (4, 4, 100, 16), (5, 3, 33, 1), (3, 5, 33, 8), (64, 16, 5000, 16), (257, 257, 700, 4),
    (2000, 31, 90, 2), (16, 16, 3000, 2), (8192, 8192, 20, 4), (0, 3, 40, 16), (3, 0, 0, 16)])
@pytest.mark.parametrize("in_place", [False, True])
def test_fork_matches_the_plain_loop(children, rows, cached, page, in_place):
    wsw = need_gpu()
    g = np.random.default_rng(children + rows + cached)
    seq, table, free = _rows(g, rows, cached, page)
    parent = g.integers(-1, max(rows, 0), children) if rows else np.full(children, -1)
    free = np.arange(children + 3) + 10 ** 6
    want = _fork(wsw, parent, seq, free, 2, table, page, in_place)
    assert want[4] == 0


@pytest.mark.parametrize("what", ["parent", "length", "pages", "head", "all"])
@pytest.mark.parametrize("n", [6, 300])
@pytest.mark.parametrize("in_place", [False, True])
def test_fork_reports_what_does_not_fit(what, n, in_place):
    wsw = need_gpu()
    g = np.random.default_rng(n)
    seq, table, _ = _rows(g, n, 60, 8)
    seq[:] = seq // 8 * 8 + 3
    parent = g.integers(0, max(2, n // 3), n)
    free, head = np.arange(n) + 5000, 0
    if what in ("parent", "all"):
        parent[1], parent[3] = n, -2
    if what in ("length", "all"):
        seq[parent[0]], seq[parent[n - 1]] = -1, table.shape[1] * 8 + 1
    if what in ("pages", "all"):
        free = free[: n // 4]
    if what == "head":
        head = n + 1
    want = _fork(wsw, parent, seq, free, head, table, 8, in_place)
    assert want[4] != 0


def _cache(wsw, g, kind, pages, page, heads, dim, layout, gap=0):
    """A PagedKV with random contents and its tensors, with `gap` unused rows of head_dim between positions."""
    shape = (pages, page, heads + gap, dim) if layout == "nhd" else (pages, heads, page + gap, dim)

    def room(dtype, last):
        s = shape[:3] + (last,)
        x = torch.randint(-120, 120, s, generator=g, device="cuda", dtype=torch.int8) if dtype == torch.int8 else \
            torch.randn(s, generator=g, device="cuda").to(dtype)
        return x

    dtype = {"fp16": torch.float16, "bf16": torch.bfloat16, "q8_0": torch.int8}[kind]
    full = [room(dtype, dim) for _ in range(2)]
    if kind == "q8_0":
        full += [room(torch.float16, dim // 32) for _ in range(2)]
    view = [x[:, :, :heads] if layout == "nhd" else x[:, :, :page] for x in full]
    return wsw.PagedKV(*view, layout=layout), full


def _copied(full, entries, layout, page, heads):
    want = [x.clone() for x in full]
    for s, d, n in entries:
        for x, y in zip(want, full):
            if layout == "nhd":
                x[d, :n, :heads] = y[s, :n, :heads]
            else:
                x[d, :, :n] = y[s, :, :n]
    return want


@pytest.mark.parametrize("kind", ["fp16", "bf16", "q8_0"])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("page,heads,dim,gap", [(1, 1, 64, 0), (16, 4, 128, 0), (8, 3, 256, 2), (64, 5, 64, 1),
                                                (256, 8, 128, 0)])
def test_copy_moves_the_filled_positions(kind, layout, page, heads, dim, gap):
    wsw = need_gpu()
    g = torch.Generator(device="cuda").manual_seed(page + heads)
    n = 9
    layers = [_cache(wsw, g, kind, 2 * n + 1, page, heads, dim, layout, gap) for _ in range(3)]
    ids = torch.randperm(2 * n, generator=g, device="cuda").to(torch.int32)
    for whole in (False, True):
        fill = torch.randint(-1, page + 3, (n,), generator=g, device="cuda", dtype=torch.int32)
        src, dst = ids[:n].clone(), ids[n:].clone()
        src[2] = dst[2] = 2 * n  # onto itself
        count = 7
        entries = [(int(s), int(d), page if whole else min(max(int(f), 0), page))
                   for s, d, f in list(zip(src, dst, fill))[:count]]
        want = [_copied(full, entries, layout, page, heads) for _, full in layers]
        err = _i32([0])
        wsw.kv_page_copy(wsw.PageCopies(src, dst, None if whole else fill, _i32([count])), [kv for kv, _ in layers],
                         err_flag=err)
        for (_, full), w in zip(layers, want):
            assert all(torch.equal(x, y) for x, y in zip(full, w))
        assert int(err) == 0


def test_copy_of_many_layers_and_of_mixed_caches():
    wsw = need_gpu()
    g = torch.Generator(device="cuda").manual_seed(3)
    kinds = ["fp16", "q8_0", "bf16"]
    layers = [_cache(wsw, g, kinds[i % 3], 6 + i % 4, 8, 1 + i % 3, (64, 128, 256)[i % 3], "nhd" if i % 2 else "hnd")
              for i in range(67)]
    src, dst = _i32([0, 7, 2, -1, 1]), _i32([3, 4, 8, 5, 1 << 30])  # some lie in the larger caches only, some in none
    want = []
    for i, (kv, full) in enumerate(layers):
        ok = [(s, d, 5) for s, d in zip(src.tolist(), dst.tolist()) if 0 <= s < kv.num_pages and 0 <= d < kv.num_pages]
        want.append(_copied(full, ok, kv.layout, 8, kv.heads))
    err = _i32([0])
    wsw.kv_page_copy(wsw.PageCopies(src, dst, _i32([5] * 5), _i32([99])), [kv for kv, _ in layers], err_flag=err)
    assert int(err) == 1
    for (_, full), w in zip(layers, want):
        assert all(torch.equal(x, y) for x, y in zip(full, w))


def _compact(wsw, seq, table, page, pool, held=None, moves=0, in_place=False, opts=None):
    want = ref.compact(seq, table, page, pool, held, moves)
    table_d = _i32(table)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out_table = table_d if in_place or moves == 0 else _i32(np.full(table.shape, 55))
    copies = wsw.PageCopies(_i32(np.full(moves, 77)), _i32(np.full(moves, 77)), None, _i32([77]))
    out = wsw.KvCompact(out_table, _i32(np.full(pool, -7)), _i32([77]), copies)
    held_d = None if held is None else torch.tensor(held, dtype=torch.uint8, device="cuda")
    r = wsw.kv_page_compact(_i32(seq), table_d, page, pool, held=held_d, max_moves=moves, out=out, err_flag=err, opts=opts)
    k = len(want[3])
    assert r.head.tolist() == [want[2]] and r.copies.count.tolist() == [k] and int(err) == want[4]
    assert list(zip(r.copies.src.tolist(), r.copies.dst.tolist()))[:k] == want[3]
    assert (r.copies.src[k:] == 77).all() and (r.copies.dst[k:] == 77).all()
    assert r.free_pages.tolist() == [-7] * want[2] + want[1]
    got = r.table.cpu().numpy()
    for i, n in enumerate(map(int, seq)):
        used = ref.pages(n, page) if 0 <= n and ref.pages(n, page) <= table.shape[1] else 0
        assert np.array_equal(got[i, :used], want[0][i, :used])
        if not (in_place or moves == 0):
            assert (got[i, used:] == 55).all()
    if in_place or moves == 0:
        assert np.array_equal(got, want[0])
    return want


@pytest.mark.parametrize("rows,cached,page,spare", [
    (1, 0, 16, 3), (1, 5, 1, 0), (3, 100, 16, 40), (64, 4000, 16, 3000), (40, 300, 8, 17), (1000, 60, 4, 9000),
    (7, 9000, 1, 100000), (0, 10, 16, 5), (300, 2000, 64, 16)])
@pytest.mark.parametrize("moves", ["none", "one", "some", "all"])
@pytest.mark.parametrize("hold", [False, True])
def test_compact_matches_the_plain_loop(rows, cached, page, spare, moves, hold):
    wsw = need_gpu()
    g = np.random.default_rng(rows + cached + spare)
    seq, table, _ = _rows(g, rows, cached, page, shared=0)
    pool = table.size + spare
    table = g.permutation(pool)[: table.size].reshape(table.shape) if rows else table
    if rows > 4:
        table[2:5] = table[2]  # rows in common
    pool = max(pool, 1)
    held = (g.random(pool) < 0.1) * g.integers(1, 256, pool) if hold else None
    count = {"none": 0, "one": 1, "some": max(1, pool // 10), "all": pool}[moves]
    for in_place in (False, True):
        want = _compact(wsw, seq, table, page, pool, held, count, in_place)
        assert want[4] == 0


@pytest.mark.parametrize("rows", [5, 200])
def test_compact_reports_entries_and_lengths(rows):
    wsw = need_gpu()
    g = np.random.default_rng(rows)
    seq, table, _ = _rows(g, rows, 200, 8)
    pool = table.size
    table = g.permutation(pool).reshape(table.shape)
    seq[:] = 150
    table[1, 2], table[3, 0], table[3, 1] = -1, pool, 2 ** 31 - 1
    seq[2], seq[4] = -5, table.shape[1] * 8 + 1
    want = _compact(wsw, seq, table, 8, pool, None, pool)
    assert want[4] == 3


def test_a_step_of_fork_copy_and_compact_replays_in_a_graph():
    """In place, as a server runs it: the captured calls, replayed, do what the loops do one after another."""
    wsw = need_gpu()
    g = np.random.default_rng(5)
    n, page, pool, width = 12, 8, 400, 10
    seq = np.full(n, 45)
    table = np.full((n, width), -1)
    table[:, :6] = g.permutation(pool)[: 6 * n].reshape(n, 6)
    gen = torch.Generator(device="cuda").manual_seed(1)
    kv, full = _cache(wsw, gen, "bf16", pool, page, 2, 64, "nhd")
    lens, tab, parent = _i32(seq), _i32(table), _i32(np.zeros(n))
    free, head = _i32(np.full(pool, -1)), _i32([0])
    err, ws = _i32([0]), torch.zeros(wsw.kv_page_compact_workspace_bytes(pool), dtype=torch.uint8, device="cuda")
    fork_out = wsw.KvFork(tab, lens, head, wsw.PageCopies(*[_i32(np.zeros(n)) for _ in range(3)], _i32([0])))
    pack_out = wsw.KvCompact(tab, free, head, wsw.PageCopies(_i32(np.zeros(5)), _i32(np.zeros(5)), None, _i32([0])))

    def step():
        wsw.kv_page_compact(lens, tab, page, pool, max_moves=5, out=pack_out, err_flag=err, ws=ws, opts={"pdl": 1})
        wsw.kv_page_copy(pack_out.copies, kv, err_flag=err, opts={"pdl": 1})
        wsw.kv_page_fork(parent, lens, free, head, tab, page, out=fork_out, err_flag=err, opts={"pdl": 1})
        wsw.kv_page_copy(fork_out.copies, [kv], err_flag=err, opts={"pdl": 1})

    def plain(table, seq, par, rows):
        table, free_l, head_l, moves, _ = ref.compact(seq, table, page, pool, None, 5)
        rows = _copied([rows], [(s, d, page) for s, d in moves], "nhd", page, 2)[0]
        table, seq, head_l, cps, _ = ref.fork(par, seq, [-1] * head_l + free_l, head_l, table, page, table)
        return table, seq, _copied([rows], cps, "nhd", page, 2)[0]

    rows = full[0].clone()
    side = torch.cuda.Stream()
    graph = None
    for i in range(5):
        par = np.sort(g.integers(0, n, n)) if i else np.arange(n)
        parent.copy_(_i32(par))
        torch.cuda.synchronize()
        if i == 0:
            with torch.cuda.stream(side):
                step()
        elif i == 1:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            graph.replay()
        else:
            graph.replay()
        torch.cuda.synchronize()
        table, seq, rows = plain(table, seq, par, rows)
        assert np.array_equal(tab.cpu().numpy(), table) and lens.tolist() == seq.tolist() and int(err) == 0
        assert torch.equal(full[0], rows)


@pytest.mark.parametrize("kind", ["bf16", "q8_0"])
def test_copies_far_into_a_large_cache(kind):
    """Element offsets past 2^32 in K and V."""
    wsw = need_gpu()
    page, heads, dim = 256, 8, 128
    pages = (1 << 32) // (page * heads * dim) + 40
    shape = (pages, page, heads, dim)
    parts = [torch.empty(shape, dtype=torch.int8 if kind == "q8_0" else torch.bfloat16, device="cuda") for _ in range(2)]
    if kind == "q8_0":
        parts += [torch.empty(shape[:3] + (dim // 32,), dtype=torch.float16, device="cuda") for _ in range(2)]
    src, dst, fill = [pages - 1, 3, pages - 2], [5, pages - 3, pages - 4], [page, 100, 7]
    for x in parts:
        for p in src + dst:
            x[p] = torch.randint(-9, 9, x[p].shape, device="cuda").to(x.dtype)
    want = [[x[d].clone() for d in dst] for x in parts]
    for w, x in zip(want, parts):
        for i, (s, n) in enumerate(zip(src, fill)):
            w[i][:n] = x[s, :n]
    err = _i32([0])
    wsw.kv_page_copy(wsw.PageCopies(_i32(src), _i32(dst), _i32(fill), _i32([3])), wsw.PagedKV(*parts), err_flag=err)
    assert int(err) == 0
    for w, x in zip(want, parts):
        assert all(torch.equal(a, x[d]) for a, d in zip(w, dst))


@pytest.mark.parametrize("n,width", [(64, 300), (8192, 40), (3, 70000)])
def test_tables_with_room_between_their_rows(n, width):
    """Strided views of wider tables, whose other entries stay."""
    wsw = need_gpu()
    g = np.random.default_rng(n)
    page = 4
    wide_in, wide_out = g.integers(0, 10 ** 6, (n, width + 5)), np.full((n, width + 9), 55)
    seq, parent = g.integers(0, width * page + 1, n), g.integers(-1, n, n)
    free = np.arange(n) + 2 * 10 ** 6
    want = ref.fork(parent, seq, free, 0, wide_in[:, 2:width + 2], page, wide_out[:, 3:width + 3])
    t, o = _i32(wide_in), _i32(wide_out)
    out = wsw.KvFork(o[:, 3:width + 3], _i32(np.zeros(n)), _i32([0]),
                     wsw.PageCopies(*[_i32(np.zeros(n)) for _ in range(3)], _i32([0])))
    wsw.kv_page_fork(_i32(parent), _i32(seq), _i32(free), _i32([0]), t[:, 2:width + 2], page, out=out)
    got = o.cpu().numpy()
    assert np.array_equal(got[:, 3:width + 3], want[0]) and (got[:, :3] == 55).all() and (got[:, width + 3:] == 55).all()
    assert int(out.head) == want[2] and out.seq_len.tolist() == want[1].tolist()


def test_the_largest_pool():
    wsw = need_gpu()
    g = np.random.default_rng(0)
    pool = 1 << 22
    table = g.permutation(pool)[:200 * 1000].reshape(200, 1000)
    _compact(wsw, g.integers(0, 16001, 200), table, 16, pool, None, 1 << 20, True)


def test_two_streams_at_once():
    """Each with its own workspace and tensors."""
    wsw = need_gpu()
    g = np.random.default_rng(1)
    pool, jobs = 50000, []
    for i in range(2):
        seq, table = g.integers(0, 8000, 64), g.permutation(pool)[:64 * 500].reshape(64, 500)
        out = wsw.KvCompact(_i32(table), _i32(np.full(pool, -1)), _i32([0]),
                            wsw.PageCopies(_i32(np.zeros(pool)), _i32(np.zeros(pool)), None, _i32([0])))
        ws = torch.zeros(wsw.kv_page_compact_workspace_bytes(pool), dtype=torch.uint8, device="cuda")
        jobs.append((seq, table, _i32(seq), _i32(table), out, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for seq, table, seq_d, table_d, out, ws, stream in jobs:
            with torch.cuda.stream(stream):
                wsw.kv_page_compact(seq_d, table_d, 16, pool, max_moves=pool, out=out, ws=ws)
    torch.cuda.synchronize()
    for seq, table, _, _, out, _, _ in jobs:
        want = ref.compact(seq, table, 16, pool, None, pool)
        got = out.table.cpu().numpy()
        for r, n in enumerate(seq):
            k = ref.pages(int(n), 16)
            assert np.array_equal(got[r, :k], want[0][r, :k])
        assert int(out.head) == want[2] and out.free_pages.tolist()[want[2]:] == want[1]
