"""Attention over shared prefixes on the GPU against the formula in 64 bits.

Tolerance.  A score's error, in units of the largest sum A = scale sum |q k| of the request: q's parts
(exact in q's own type, for fp16 over bf16 and for fp32 over bf16 pages within a prefix; 2^-22 over binary16;
2^-17 for fp32 or fp16 over bf16 in the rest, which the paged attention has, but exact there too under fp32),
parts * head_dim / 16 + 2 fp32 sums and products (2^-23 each: tensor-core sums may cut), softcap's tanh
(7 2^-24 of softcap), the slope's product and sum (2^-22 of slope distance), the exponential (2^-22).  A relative
error e of every weight moves an output by at most 2 e times its weighted magnitude M = sum w |v| / sum w.
Under 16-bit queries a weight is rounded once, U = 2^-8 (bf16 cache) or 2^-11 of itself, and binary16 weights
are off by 2^-32 of the largest (below their normal range), n 2^-32 max |v| in sum; under fp32 queries U = 2^-22 over
binary16, 0 over bf16 (three parts).  Sums: n / 16 products' (times P's parts), 2^-23 each, a row's weights TP / 4 +
n / TP <= n / 16 + 32, and at most 160 joined pieces.  Then half a step of the output's type.
lse: the score error, 2^-22, the sums, and 2^-22 |lse|."""
import math

import numpy as np
import pytest
import torch

import kv_share_ref as ref
from helpers import need_gpu

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
STEP = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
TYPES = [("fp32", "fp16"), ("fp32", "q8_0"), ("fp32", "bf16"), ("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "q8_0"),
         ("bf16", "fp16"), ("fp16", "bf16"), ("fp16", "q8_0")]


class Case:
    """groups: [(prefix length, [lens of its requests])]; requests before and behind them: loose lens."""

    def __init__(self, wsw, groups, before=(), behind=(), kvh=2, group=4, d=128, q="bf16", cache="bf16", page=16, nhd=True,
                 seed=0, copies=False, qsigma=1.0, junk=float("nan")):
        g = torch.Generator().manual_seed(seed)
        self.wsw, self.kvh, self.group, self.d, self.page, self.cache, self.qt = wsw, kvh, group, d, page, cache, q
        self.lens = list(before) + [n for _, ls in groups for n in ls] + list(behind)
        n = len(self.lens)
        self.prefix = [p for p, _ in groups]
        self.cu = [len(before)]
        for _, ls in groups:
            self.cu.append(self.cu[-1] + len(ls))
        need = [-(-max(x, 0) // page) for x in self.lens]
        width = max(need + [1]) + 1
        self.table = torch.full((n, width), -1, dtype=torch.int64)
        used_pages, share = 0, []
        for r, k in enumerate(need):
            self.table[r, :k] = torch.arange(used_pages, used_pages + k)
            used_pages += k
        for i, (p, ls) in enumerate(groups):  # the group's whole prefix pages in common, its last one a copy
            rows = range(self.cu[i], self.cu[i + 1])
            full = [r for r in rows if self.lens[r] >= p]
            for r in full[1:]:
                if not copies:
                    self.table[r, :p // page] = self.table[full[0], :p // page]
                share.append((full[0], r, p if copies else p % page, 0 if copies else p // page * page))
        perm = torch.randperm(used_pages + 3, generator=g)
        self.table = torch.where(self.table >= 0, perm[self.table.clamp(min=0)], -1)
        pages = len(perm)
        if cache == "q8_0":
            codes = torch.randint(-127, 128, (2, pages * page, kvh, d), generator=g).to(torch.int8)
            scales = ((torch.rand(2, pages * page, kvh, d // 32, generator=g) + 1.5) / 127).half()
            parts = [codes, scales]
        else:
            parts = [torch.randn(2, pages * page, kvh, d, generator=g).to(DT[cache])]
        for a, r, count, start in share:
            for x in parts:
                x[:, self.slots(r, start, start + count)] = x[:, self.slots(a, start, start + count)]
        used = torch.zeros(pages * page, dtype=torch.bool)
        for r, x in enumerate(self.lens):
            if x > 0:
                used[self.slots(r, 0, x)] = True
        if cache == "q8_0":
            self.vals = (codes.double() * scales.double().repeat_interleave(32, -1)).half().double().numpy()
            scales[:, ~used] = junk
        else:
            self.vals = parts[0].double().numpy()
            parts[0] = parts[0].clone()
            parts[0][:, ~used] = junk
        self.q = (torch.randn(n, kvh * group, d, generator=g) * qsigma).to(DT[q])

        def paged(t):
            t = t.reshape(pages, page, kvh, -1)
            return (t if nhd else t.transpose(1, 2).contiguous()).cuda()
        both = [paged(x[i]) for x in parts for i in range(2)]
        self.kv = wsw.PagedKV(*both, layout="nhd" if nhd else "hnd")
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table_d, self.lens_d = self.table.to(torch.int32).cuda(), torch.tensor(self.lens, **i32)
        self.cu_d, self.prefix_d = torch.tensor(self.cu, **i32), torch.tensor(self.prefix, **i32)

    def slots(self, r, a, b):
        p = torch.arange(a, b)
        return self.table[r, p // self.page] * self.page + p % self.page

    def run(self, scale=None, **kw):
        n = len(self.lens)
        lse = torch.full((n, self.kvh * self.group), 7.0, device="cuda")
        out = torch.full((n, self.kvh * self.group, self.d), 7.0, device="cuda", dtype=DT[self.qt])
        self.wsw.attn_paged_prefix(self.q.cuda(), self.kv, self.table_d, self.lens_d, self.cu_d, self.prefix_d, scale=scale,
                                   lse=lse, out=out, **{"share": True, **kw})
        return out, lse

    def check(self, scale=None, softcap=0.0, slopes=None, hidden=None, **kw):
        """hidden: {request: positions that a bad table entry hides}.  Where a group's rows would fill two row tiles, a
        second time in a table with room for rows so long that they do."""
        rows, narrow = len(self.lens) * self.group, self.table_d
        if rows > 128 * len(self.prefix) and kw.get("share", True):
            width = (21 * 152 * 128 // (self.kvh * (rows // 128)) + 128) // self.page + 1
            if width > narrow.shape[1]:
                self.table_d = torch.full((len(self.lens), width), -1, dtype=torch.int32, device="cuda")
                self.table_d[:, :narrow.shape[1]] = narrow
                self._check(scale, softcap, slopes, hidden, **kw)
                self.table_d = narrow
        return self._check(scale, softcap, slopes, hidden, **kw)

    def _check(self, scale, softcap, slopes, hidden, **kw):
        scale = 1 / math.sqrt(self.d) if scale is None else scale
        sl = None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda")
        out, lse = self.run(scale, softcap=softcap, slopes=sl, **kw)
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        q = self.q.double().numpy()
        half, wide = self.cache == "bf16", self.qt == "fp32"
        for r, n in enumerate(self.lens):
            p = np.array([x for x in range(max(n, 0)) if x not in (hidden or {}).get(r, ())], dtype=np.int64)
            if len(p) == 0:
                assert (got[r] == 0).all() and (gl[r] == -math.inf).all(), r
                continue
            rows = self.table[r].numpy()[p // self.page] * self.page + p % self.page
            dist = (n - 1 - p).astype(np.float64)
            fs = None if slopes is None else np.asarray(slopes, np.float32).astype(np.float64)
            k, v = self.vals[0][rows], self.vals[1][rows]
            want, wl, mag = ref.attend(q[r], k, v, scale, softcap, fs, dist)
            a = abs(scale) * max(float((np.abs(q[r].reshape(self.kvh, self.group, -1)[h]) @ np.abs(k[:, h]).T).max())
                                 for h in range(self.kvh))
            exact = self.qt == ("bf16" if half else "fp16") or wide and half
            parts = 3 if wide and half else 2 if wide or half and self.qt == "fp16" else 1
            e = a * ((0 if exact else 2.0 ** -17 if half else 2.0 ** -22) + (parts * self.d / 16 + 2) * 2.0 ** -23)
            e += softcap * 7 * 2.0 ** -24 + (0 if fs is None else fs.max() * dist.max() * 2.0 ** -22) + 2.0 ** -22
            u = (0 if half else 2.0 ** -22) if wide else 2.0 ** -8 if half else 2.0 ** -11
            sums = (len(p) / 16 * parts + 32 + 160) * 2.0 ** -23
            lim = mag * (2 * e + u + sums) + (0 if half else len(p) * 2.0 ** -32 * np.abs(v).max())
            assert np.isfinite(got[r]).all(), r
            bad = np.abs(got[r] - want) - (lim + STEP[self.qt] * (np.abs(want) + lim) + 2.0 ** -25)
            assert (bad <= 0).all(), "request %d (length %d): over by %.3g" % (r, n, bad.max())
            lim = e + 2.0 ** -22 + sums + 2.0 ** -22 * np.abs(wl)
            assert (np.abs(gl[r] - wl) <= lim).all(), "request %d: lse off by %.3g" % (r, np.abs(gl[r] - wl).max())
        return out, lse


def _lens(prefix, *rest):
    return [prefix + x for x in rest]


@pytest.mark.parametrize("q,cache", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("per,group", [(3, 4), (20, 10)])
def test_types_and_row_tiles(q, cache, d, per, group):
    wsw = need_gpu()
    g = np.random.default_rng(per)
    c = Case(wsw, [(700, [700 + int(x) for x in g.integers(0, 90, per)]), (333, _lens(333, 1, 40))], kvh=2, group=group, d=d,
             q=q, cache=cache, nhd=per == 3, page=16)
    c.check()


@pytest.mark.parametrize("prefix", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 5000])
@pytest.mark.parametrize("page", [1, 8, 64, 256])
@pytest.mark.parametrize("q,cache", [("bf16", "bf16"), ("fp32", "q8_0")])
def test_prefix_lengths_and_pages(prefix, page, q, cache):
    wsw = need_gpu()
    Case(wsw, [(prefix, _lens(prefix, 0, 1, 17, 200))], page=page, kvh=1, group=8, q=q, cache=cache, seed=prefix).check()


@pytest.mark.parametrize("per,group", [(2, 1), (2, 64), (5, 3), (16, 8), (17, 8), (33, 8), (100, 4), (257, 1), (40, 40)])
@pytest.mark.parametrize("q,cache", [("fp16", "fp16"), ("fp32", "bf16")])
def test_rows_of_a_group(per, group, q, cache):
    wsw = need_gpu()
    Case(wsw, [(300, [300 + i % 7 for i in range(per)])], kvh=1 if group > 8 else 3, group=group, d=64, q=q, cache=cache,
         seed=per).check()


def test_many_groups_of_all_sizes():
    wsw = need_gpu()
    g = np.random.default_rng(0)
    groups = []
    for i in range(60):
        p = int(g.integers(1, 600))
        groups.append((p, [p + int(x) for x in g.integers(0, 50, int(g.integers(0, 9)))]))
    Case(wsw, groups, before=[3, 0, 200], behind=[77, 1], kvh=2, group=3, d=64, q="fp16", cache="fp16").check()
    Case(wsw, groups, kvh=1, group=5, d=128, q="fp32", cache="q8_0", page=8).check()


@pytest.mark.parametrize("q,cache", [("bf16", "bf16"), ("fp32", "fp16")])
@pytest.mark.parametrize("copies", [False, True])
def test_short_requests_unused_rows_and_loose_ones(q, cache, copies):
    """Requests shorter than the prefix, empty ones (first of the group, too), groups of one and none."""
    wsw = need_gpu()
    c = Case(wsw, [(200, [0, 150, 230, 200, 199, 300]), (64, [64]), (90, []), (100, [0, 0, 5]), (0, [7, 9]), (50, [90, 60, 55])],
             before=[10, 0], behind=[33], kvh=2, group=4, q=q, cache=cache, copies=copies)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(err_flag=err)
    assert int(err) == 0


@pytest.mark.parametrize("q,cache", [("bf16", "bf16"), ("fp32", "q8_0"), ("fp16", "fp16")])
def test_softcap_slopes_and_scales(q, cache):
    wsw = need_gpu()
    c = Case(wsw, [(500, _lens(500, 3, 60, 90, 1)), (130, _lens(130, 5, 5))], kvh=2, group=4, q=q, cache=cache, qsigma=3.0)
    c.check(softcap=5.0)
    c.check(slopes=[2.0 ** -(i + 1) for i in range(8)])
    c.check(softcap=20.0, slopes=[0.0, 0.5] * 4)
    c.check(scale=-0.05)
    c.check(scale=0.0)
    c.check(scale=1.0)
    c.check(softcap=3e38)


@pytest.mark.parametrize("q,cache,sigma", [("fp32", "fp16", 1e6), ("fp32", "fp16", 1e-9), ("bf16", "fp16", 1e7),
                                           ("bf16", "q8_0", 1e-12), ("fp32", "bf16", 1e12), ("bf16", "bf16", 1e-20)])
def test_queries_of_any_size(q, cache, sigma):
    wsw = need_gpu()
    c = Case(wsw, [(300, _lens(300, 1, 60, 7))], kvh=2, group=4, q=q, cache=cache, qsigma=sigma)
    c.q[0, 3] = 0
    c.check(scale=1 / sigma / math.sqrt(128))


@pytest.mark.parametrize("cache", ["bf16", "q8_0"])
@pytest.mark.parametrize("page", [1, 16])
def test_bad_table_entries_hide_their_positions(cache, page):
    wsw = need_gpu()
    c = Case(wsw, [(400, _lens(400, 10, 33)), (48, _lens(48, 3, 3))], kvh=1, group=4, page=page, cache=cache)
    hidden = {}
    for r, entry, what in ((0, 3, -1), (0, 7, 10 ** 6), (2, 0, -5), (2, 1, 1 << 30), (2, 2, -1)):
        c.table_d[r, entry] = what
        for x in (0, 1) if r == 0 else (2, 3):  # the prefix is read through the first request's row
            hidden.setdefault(x, set()).update(range(entry * page, (entry + 1) * page))
    if page == 1:
        hidden[2] -= set(range(48, 51))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(hidden=hidden, err_flag=err)
    assert int(err) == 1


def test_bounds_that_do_not_ascend_are_moved():
    """Descending and far bounds: every request is still attended once, and bit 2 says so."""
    wsw = need_gpu()
    for cu, prefix in (([0, 4, 2, 6], [100, 100, 100]), ([-3, 3, 3, 1000], [100, 5, 100]), ([0, 2, 4, 6], [100, -1, 10 ** 9]),
                       ([6, 0, 0, 0], [100, 100, 100]), ([-1, -1, -1, -1], [9, 9, 9])):
        c = Case(wsw, [(100, _lens(100, 1, 2, 3, 40, 50, 60))], kvh=2, group=4)
        c.cu_d = torch.tensor(cu, dtype=torch.int32, device="cuda")
        c.prefix_d = torch.tensor(prefix, dtype=torch.int32, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        c.check(err_flag=err)
        assert int(err) == 4


@pytest.mark.parametrize("q,cache", [("bf16", "bf16"), ("fp32", "fp16"), ("fp32", "bf16")])
def test_a_long_prefix(q, cache):
    wsw = need_gpu()
    Case(wsw, [(20000, _lens(20000, 1, 300, 40, 0, 5))], kvh=1, group=4, q=q, cache=cache, page=64).check()


def test_one_workspace_graphs_streams_and_repeated_calls():
    wsw = need_gpu()
    cases = [Case(wsw, [(300, _lens(300, *range(20)))], kvh=2, group=8, q="bf16", cache="bf16"),
             Case(wsw, [(90, _lens(90, 4, 9)), (40, _lens(40, 1, 2, 3))], kvh=3, group=5, d=64, q="fp32", cache="q8_0"),
             Case(wsw, [(700, _lens(700, 100, 200))], kvh=1, group=2, q="fp16", cache="fp16")]
    need = max(wsw.attn_paged_prefix_workspace_bytes(len(c.lens), len(c.prefix), c.kvh * c.group, c.kvh, c.d) for c in cases)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    want = [c.check() for c in cases]
    for turn in range(2):
        for c, (out, lse) in zip(cases, want):
            o, l = c.run(ws=ws, opts={"pdl": turn})
            assert torch.equal(o, out) and torch.equal(l, lse)
    assert (ws[:2048] == 0).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, l = cases[0].run(ws=ws)
    side.synchronize()
    assert torch.equal(o, want[0][0]) and torch.equal(l, want[0][1])
    c = cases[1]
    q, out, lse = c.q.cuda(), torch.empty_like(want[1][0]), torch.empty_like(want[1][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wsw.attn_paged_prefix(q, c.kv, c.table_d, c.lens_d, c.cu_d, c.prefix_d, out=out, lse=lse, ws=ws, share=True)
    for _ in range(3):
        out.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[1][0]) and torch.equal(lse, want[1][1])


@pytest.mark.parametrize("q,cache", [("bf16", "bf16"), ("fp32", "q8_0")])
def test_a_small_batch_goes_the_paged_way(q, cache):
    """Without `share` the result is attn_paged_decode's, bit for bit, and the groups are not looked at."""
    wsw = need_gpu()
    c = Case(wsw, [(300, _lens(300, 1, 60, 7))], kvh=2, group=4, q=q, cache=cache)
    c.cu_d.fill_(77)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c.check(share=False, err_flag=err)
    want_lse = torch.empty_like(lse)
    want = wsw.attn_paged_decode(c.q.cuda(), c.kv, c.table_d, c.lens_d, lse=want_lse)
    assert torch.equal(out, want) and torch.equal(lse, want_lse) and int(err) == 0


def test_a_large_batch_is_shared():
    """A block table of more than 128 MB of positions, all but the first few unused."""
    wsw = need_gpu()
    c = Case(wsw, [(300, _lens(300, 1, 60, 7))], kvh=2, group=4, page=16)
    wide = torch.full((3, 1 << 16), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.table_d.shape[1]] = c.table_d
    small, _ = c.check()
    c.table_d = wide
    out, _ = c.check(share=False)
    assert torch.equal(out, small)


@pytest.mark.parametrize("q,cache", [("bf16", "bf16"), ("fp32", "q8_0"), ("fp32", "bf16"), ("fp16", "fp16")])
@pytest.mark.parametrize("prefix", [1, 40, 64, 128])
def test_pieces_of_one_tile(q, cache, prefix):
    """Several pieces of one tile (two, of 64 positions) to a block: a ring place of the first tiles belongs
    to a later piece, whose queries come while the loads of the one before may still be behind."""
    c = Case(need_gpu(), [(prefix, _lens(prefix, 0, 1))] * 400, d=64, q=q, cache=cache, group=2)
    out, lse = c.check()
    for _ in range(20):
        o, l = c.run()
        assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("cache", ["bf16", "q8_0"])
def test_pages_far_into_a_large_cache(cache):
    """Element offsets past 2^32 in K and V: the same result as in a small cache."""
    wsw = need_gpu()
    c = Case(wsw, [(600, _lens(600, 0, 30, 1))], kvh=8, group=4, page=256, q="bf16", cache=cache, junk=0.0)
    want, want_lse = c.check()
    pages = (1 << 32) // (256 * 8 * 128) + 2
    few = c.kv.num_pages
    small = [x for x in (c.kv.k, c.kv.v, c.kv.kd, c.kv.vd) if x is not None]
    big = [torch.empty((pages + few,) + tuple(x.shape[1:]), dtype=x.dtype, device="cuda") for x in small]
    for b, x in zip(big, small):
        b[pages:] = x
    c.kv = wsw.PagedKV(*big)
    c.table_d = torch.where(c.table_d >= 0, c.table_d + pages, c.table_d)
    out, lse = c.run()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_two_streams_at_once():
    """Each call with its own workspace: the results of calls alone."""
    wsw = need_gpu()
    cases = [Case(wsw, [(3000, _lens(3000, *range(24)))], kvh=4, group=8, q="bf16", cache="bf16", seed=s) for s in (1, 2)]
    want = [c.run() for c in cases]
    ws = [torch.zeros(wsw.attn_paged_prefix_workspace_bytes(24, 1, 32, 4, 128), dtype=torch.uint8, device="cuda") for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    qs = [c.q.cuda() for c in cases]
    outs = [torch.empty_like(w[0]) for w in want]
    torch.cuda.synchronize()
    for _ in range(30):
        for c, q, o, w, s in zip(cases, qs, outs, ws, streams):
            with torch.cuda.stream(s):
                wsw.attn_paged_prefix(q, c.kv, c.table_d, c.lens_d, c.cu_d, c.prefix_d, out=o, ws=w, share=True)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w[0]) for o, w in zip(outs, want))


@pytest.mark.parametrize("groups", [1, 15, 16, 17, 20, 60, 160, 5000])
@pytest.mark.parametrize("q,cache", [("bf16", "bf16"), ("fp32", "fp16")])
def test_short_tables_of_many_groups(groups, q, cache):
    """Fewer tiles than SMs, whose pieces still have their places in the list."""
    c = Case(need_gpu(), [(20 + g % 13, _lens(20 + g % 13, 0, 2)) for g in range(groups)], kvh=1, group=1, d=64, q=q, cache=cache)
    assert c.table.shape[1] * c.page <= 64
    c.check()


@pytest.mark.parametrize("q,cache,d", [("bf16", "bf16", 128), ("fp16", "fp16", 64), ("bf16", "q8_0", 128)])
def test_both_row_tilings(q, cache, d):
    """More than 128 rows of a group, with cap, slopes and a negative scale."""
    c = Case(need_gpu(), [(700, _lens(700, *range(40))), (1300, _lens(1300, *range(3)))], kvh=2, group=8, d=d, q=q, cache=cache)
    c.check()
    c.check(-0.2, softcap=20.0)
    c.check(softcap=30.0, slopes=[2.0 ** -(i % 8 + 1) for i in range(16)])
