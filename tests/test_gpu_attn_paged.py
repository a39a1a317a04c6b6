"""Paged decode attention on the GPU against the formula in 64 bits.

Tolerance.  A score's error, in units of the largest sum A = scale sum |q k| of the request:
q as high part and residual (Q = 2^-22 with binary16, 2^-17 with bf16, 0 for a 16-bit q of the
cache's own type), head_dim / 16 + 2 fp32 sums and products (2^-23 each: tensor-core sums may
cut), softcap's tanh (2^-22 of softcap), the slope's product and sum (2^-23 of slope
distance), and in log2 units the exponential (2^-22).  A relative error e of every weight
moves an output by at most 2 e times its weighted magnitude M = sum w |v| / sum w; the weights'
rounding is Q' = 2^-22 (bf16 2^-17), and a warp adds at most `tiles` products, 2^-23 each.
Then half a step of the output's type.  lse: the score error, 2^-22 + tiles 2^-23 for the sum
and 2^-22 |lse|."""
import math

import numpy as np
import pytest
import torch

import kv_step_ref as ref
from helpers import need_gpu

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
STEP = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}


class Case:
    """Inputs of one call, and its check."""

    def __init__(self, wsw, lens, kvh=2, group=4, d=128, q="fp32", cache="fp16", page=16, nhd=True, seed=0, qsigma=1.0,
                 extra=3, junk=float("nan")):
        g = torch.Generator().manual_seed(seed)
        self.wsw, self.kvh, self.group, self.d, self.page, self.cache, self.qt = wsw, kvh, group, d, page, cache, q
        self.lens = list(lens)
        n = len(self.lens)
        need = [-(-max(x, 0) // page) for x in self.lens]
        width = max(need + [1]) + 1
        ids = torch.randperm(sum(need) + extra, generator=g)
        pages = len(ids)
        self.table = torch.full((n, width), -1, dtype=torch.int64)
        at = 0
        for r, k in enumerate(need):
            self.table[r, :k] = ids[at: at + k]
            at += k
        # rows by slot; whatever no request owns is junk that must never be used
        if cache == "q8_0":
            codes = torch.randint(-127, 128, (2, pages * page, kvh, d), generator=g).to(torch.int8)
            scales = ((torch.rand(2, pages * page, kvh, d // 32, generator=g) + 1.5) / 127).half()
            vals = (codes.double() * scales.double().repeat_interleave(32, -1)).half()
        else:
            vals = torch.randn(2, pages * page, kvh, d, generator=g).to(DT[cache])
        used = torch.zeros(pages * page, dtype=torch.bool)
        for r, x in enumerate(self.lens):
            if x > 0:
                used[self.slots(r, 0, x)] = True
        self.vals = vals.double().numpy()
        self.q = (torch.randn(n, kvh * group, d, generator=g) * qsigma).to(DT[q])
        if cache == "q8_0":
            scales[:, ~used] = junk
            arr, sc = codes, scales
        else:
            vals = vals.clone()
            vals[:, ~used] = junk
            arr, sc = vals, None

        def paged(t):
            t = t.reshape(pages, page, kvh, -1)
            return (t if nhd else t.transpose(1, 2).contiguous()).cuda()
        self.kv = wsw.PagedKV(paged(arr[0]), paged(arr[1]), *((paged(sc[0]), paged(sc[1])) if sc is not None else
                                                              (None, None)), layout="nhd" if nhd else "hnd")
        self.table_d = self.table.to(torch.int32).cuda()
        self.lens_d = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def slots(self, r, a, b):
        p = torch.arange(a, b)
        return self.table[r, p // self.page] * self.page + p % self.page

    def run(self, scale=None, **kw):
        n = len(self.lens)
        lse = torch.full((n, self.kvh * self.group), 7.0, device="cuda")
        out = self.wsw.attn_paged_decode(self.q.cuda(), self.kv, self.table_d, self.lens_d, scale=scale, lse=lse, **kw)
        return out, lse

    def check(self, scale=None, softcap=0.0, window=0, slopes=None, hidden=None, **kw):
        """hidden: {request: positions that a bad table entry hides}."""
        scale = 1 / math.sqrt(self.d) if scale is None else scale
        sl = None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda")
        out, lse = self.run(scale, softcap=softcap, window=window, slopes=sl, **kw)
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        q = self.q.double().numpy()
        for r, n in enumerate(self.lens):
            a = max(0, n - window) if window else 0
            p = np.array([x for x in range(a, max(n, 0)) if x not in (hidden or {}).get(r, ())], dtype=np.int64)
            if len(p) == 0:
                assert (got[r] == 0).all() and (gl[r] == -math.inf).all(), r
                continue
            rows = (self.table[r].numpy()[p // self.page] * self.page + p % self.page)
            dist = (n - 1 - p).astype(np.float64)
            fs = None if slopes is None else np.asarray(slopes, np.float32).astype(np.float64)
            want, wl, mag, terms = ref.attend(q[r], self.vals[0][rows], self.vals[1][rows], scale, softcap, fs, dist)
            half = self.cache == "bf16"
            exact_q = self.qt == ("bf16" if half else "fp16")
            e = terms * ((0 if exact_q else 2.0 ** -17 if half else 2.0 ** -22) + (self.d / 16 + 2) * 2.0 ** -23)
            e += softcap * 2.0 ** -22 + (0 if fs is None else fs.max() * dist.max() * 2.0 ** -22) + 2.0 ** -22
            tiles = len(p) / 16 + 1
            lim = mag * (2 * e + (2.0 ** -17 if half else 2.0 ** -22) + tiles * 2.0 ** -23)
            assert np.isfinite(got[r]).all(), r
            bad = np.abs(got[r] - want) - (lim + STEP[self.qt] * (np.abs(want) + lim) + 2.0 ** -25)
            assert (bad <= 0).all(), "request %d (length %d): over by %.3g" % (r, n, bad.max())
            lim = e + 2.0 ** -22 + tiles * 2.0 ** -23 + 2.0 ** -22 * np.abs(wl)
            assert (np.abs(gl[r] - wl) <= lim).all(), "request %d: lse off by %.3g" % (r, np.abs(gl[r] - wl).max())
        return out, lse


TYPES = [("fp32", "fp16"), ("fp32", "q8_0"), ("fp32", "bf16"), ("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "q8_0"),
         ("bf16", "fp16"), ("fp16", "bf16")]


@pytest.mark.parametrize("q,cache", TYPES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 8, 10])
def test_types_widths_and_groups(q, cache, d, group):
    wsw = need_gpu()
    Case(wsw, [1, 16, 100, 0, 333], kvh=2, group=group, d=d, q=q, cache=cache, nhd=group != 8).check()


@pytest.mark.parametrize("group", [2, 3, 4, 5, 7, 9, 12, 16, 17, 40])
def test_every_group(group):
    wsw = need_gpu()
    Case(wsw, [1, 50, 300], kvh=3, group=group, seed=group).check()
    Case(wsw, [40, 129], kvh=1, group=group, cache="q8_0", seed=group).check()


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 127, 128, 129, 1000, 2048, 4097])
@pytest.mark.parametrize("page", [1, 8, 16, 64, 4096])
def test_lengths_and_pages(length, page):
    wsw = need_gpu()
    Case(wsw, [length], page=page, kvh=1, group=8, seed=length).check()
    Case(wsw, [length, 3, length], page=page, kvh=2, group=2, cache="q8_0", nhd=False, seed=length).check()


@pytest.mark.parametrize("cache", ["fp16", "bf16", "q8_0"])
def test_long_requests(cache):
    wsw = need_gpu()
    Case(wsw, [32768], kvh=2, group=4, cache=cache, q="bf16" if cache == "bf16" else "fp32").check()


def test_ragged_batches():
    wsw = need_gpu()
    g = np.random.default_rng(0)
    lens = [int(x) for x in g.integers(0, 700, 150)]
    Case(wsw, lens, kvh=4, group=8, page=32).check()
    Case(wsw, [5] * 400 + [3000] + [0] * 30 + [17] * 7, kvh=1, group=2, d=64, page=8, q="fp16").check()
    Case(wsw, [0, 0, 0], kvh=1, group=2).check()
    Case(wsw, [1] * 700, kvh=2, group=1, cache="q8_0").check()
    Case(wsw, [2000, 0, 1, 2000], kvh=4, group=16, d=256, cache="bf16", q="bf16").check()


@pytest.mark.parametrize("seed", range(6))
def test_lists_of_long_and_short_requests(seed):
    """Lists long enough for every rule of their cutting: pairs shared by many CTAs, cuts near
    a long pair's ends, short pairs kept whole, requests of no tokens between them."""
    wsw = need_gpu()
    g = np.random.default_rng(100 + seed)
    lens = [int(math.exp(x)) for x in g.uniform(0, math.log(9000), 24)] + [int(g.integers(5000, 16000)), 0]
    g.shuffle(lens)
    cache, q = [("fp16", "fp32"), ("q8_0", "fp32"), ("bf16", "bf16")][seed % 3]
    Case(wsw, lens, kvh=[3, 4, 8][seed // 2], group=[4, 8, 10][(seed // 3) % 3], cache=cache, q=q,
         page=[16, 64, 8][seed % 3], nhd=seed % 2 == 0, seed=seed).check()


@pytest.mark.parametrize("window", [1, 15, 16, 100, 5000])
def test_windows(window):
    wsw = need_gpu()
    Case(wsw, [1, 16, 101, 999, 0, 4000], seed=window).check(window=window)
    Case(wsw, [120, 2047], cache="q8_0", page=8, group=10, seed=window).check(window=window)


@pytest.mark.parametrize("cache", ["fp16", "q8_0"])
@pytest.mark.parametrize("group", [4, 12])
def test_softcap_slopes_and_scale(cache, group):
    wsw = need_gpu()
    c = Case(wsw, [1, 40, 700, 3001], kvh=2, group=group, cache=cache, qsigma=3.0)
    slopes = [2.0 ** (-8 * (i + 1) / (2 * group)) for i in range(2 * group)]
    c.check(softcap=30.0)
    c.check(slopes=slopes)
    c.check(softcap=5.0, slopes=slopes, window=500, scale=0.3)
    c.check(scale=0.0)
    c.check(scale=-0.05)


def test_large_scores_stay_finite():
    wsw = need_gpu()
    Case(wsw, [500, 1000], qsigma=40.0).check()


@pytest.mark.parametrize("q", ["fp32", "bf16"])
@pytest.mark.parametrize("cache,d", [("fp16", 128), ("q8_0", 64), ("fp16", 256), ("bf16", 128), ("q8_0", 128)])
@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e6, 1e30])
@pytest.mark.parametrize("softcap", [0.0, 2.0])
def test_queries_of_any_size(q, cache, d, size, softcap):
    """q far outside binary16's range, the scale the other way: ordinary scores."""
    wsw = need_gpu()
    Case(wsw, [70, 3], group=10, d=d, q=q, cache=cache, qsigma=size).check(scale=1 / (math.sqrt(d) * size),
                                                                         softcap=softcap)


def test_a_zero_query_and_one_of_another_size_share_a_head():
    wsw = need_gpu()
    c = Case(wsw, [300, 17, 1], group=4)
    c.q[:, 0] = 0.0
    c.q[:, 1] *= 2.0 ** 30
    c.q[:, 6] *= 2.0 ** -40
    c.check(scale=2.0 ** -30)


def test_bad_pages_are_hidden_and_flagged():
    wsw = need_gpu()
    c = Case(wsw, [100, 64, 40], page=16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(err_flag=err)
    assert int(err) == 0
    c.table_d[0, 2] = c.kv.num_pages       # positions 32 .. 47
    c.table_d[1, 0] = -5                   # positions 0 .. 15
    c.table_d[2, :] = 1 << 30              # all of it
    c.check(err_flag=err, hidden={0: range(32, 48), 1: range(16), 2: range(40)})
    assert int(err) == 1


def test_lengths_outside_the_table_are_cut_and_flagged():
    wsw = need_gpu()
    c = Case(wsw, [100, 50], page=16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.lens_d[1] = -7
    c.lens = [100, 0]
    c.check(err_flag=err)
    assert int(err) == 2
    c = Case(wsw, [128, 64], page=16)
    c.table_d = c.table_d[:, :8].contiguous()
    c.lens_d[0] = 5000  # 8 pages of 16: 128 positions
    err.zero_()
    c.check(err_flag=err)
    assert int(err) == 2


def test_strided_cache_and_table():
    """K and V interleaved in one buffer, rows padded, a table with a longer row."""
    wsw = need_gpu()
    c = Case(wsw, [70, 33], page=16, kvh=2)
    pages = c.kv.num_pages
    buf = torch.full((pages, 2, 16, 2, 136), float("nan"), dtype=torch.float16, device="cuda")
    buf[:, 0, :, :, :128] = c.kv.k
    buf[:, 1, :, :, :128] = c.kv.v
    c.kv = wsw.PagedKV(buf[:, 0, :, :, :128], buf[:, 1, :, :, :128])
    wide = torch.full((2, c.table_d.shape[1] + 9), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :c.table_d.shape[1]] = c.table_d
    c.table_d = wide[:, :c.table_d.shape[1]]
    c.check()


def test_options_repeats_streams_and_graphs_change_no_bit():
    wsw = need_gpu()
    c = Case(wsw, [3000, 5, 700, 0, 1234], kvh=4, group=8)
    ws = torch.zeros(wsw.attn_paged_decode_workspace_bytes(5, 32, 4, 128), dtype=torch.uint8, device="cuda")
    a, la = c.check(ws=ws)
    other = Case(wsw, [64, 65, 4000], kvh=2, group=3, seed=9)
    for opts in (None, {"pdl": 1}, {"ctas_per_sm": 2}):
        other.check(ws=ws, opts=opts)
        b, lb = c.run(ws=ws, opts=opts)
        assert torch.equal(a, b) and torch.equal(la, lb)
    torch.cuda.synchronize()
    assert int(ws[:2048].view(torch.int32).abs().sum()) == 0, "counters left nonzero"
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b, lb = c.run()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, b) and torch.equal(la, lb)
    q, out, lse = c.q.cuda(), torch.empty_like(a), torch.empty_like(la)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wsw.attn_paged_decode(q, c.kv, c.table_d, c.lens_d, out=out, lse=lse, ws=ws)
    for lens in ([3000, 5, 700, 0, 1234], [1, 0, 16, 0, 40]):
        c.lens_d.copy_(torch.tensor(lens))
        graph.replay()
        c.lens = lens
        b, lb = c.check(ws=ws)
        assert torch.equal(out, b) and torch.equal(lse, lb)


def test_layouts_agree_bit_for_bit():
    wsw = need_gpu()
    for cache in ("fp16", "q8_0"):
        a = Case(wsw, [300, 77], cache=cache, nhd=True, seed=3)
        b = Case(wsw, [300, 77], cache=cache, nhd=False, seed=3)
        assert torch.equal(a.run()[0], b.run()[0])


def test_equals_the_contiguous_decode_attention():
    """One request whose pages lie in order is the contiguous call's input, too."""
    wsw = need_gpu()
    g = torch.Generator().manual_seed(8)
    n, kvh, group = 1500, 4, 8
    k = torch.randn(n, kvh, 128, generator=g).half().cuda()
    v = torch.randn(n, kvh, 128, generator=g).half().cuda()
    q = torch.randn(kvh, group, 128, generator=g).cuda()
    pad = -n % 16
    pk, pv = (torch.cat([x, x.new_zeros(pad, kvh, 128)]).view(-1, 16, kvh, 128) for x in (k, v))
    table = torch.arange(pk.shape[0], dtype=torch.int32, device="cuda")[None]
    a = wsw.attn_decode_f16(q, k.permute(1, 0, 2), v.permute(1, 0, 2))
    b = wsw.attn_paged_decode(q.view(1, 32, 128), wsw.PagedKV(pk, pv), table,
                              torch.tensor([n], dtype=torch.int32, device="cuda"))
    assert (a.view(1, 32, 128) - b).abs().max() <= 2e-4 * b.abs().max()  # each is within 1e-4 of the formula
