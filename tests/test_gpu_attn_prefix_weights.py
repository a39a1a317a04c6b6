"""Attention over shared prefixes keeps the bits of its softmax weights that attn_paged_decode keeps.

Values come in pairs of opposite sign at positions of nearly the same key, so that the result is a small
difference of weights: their rounding shows, the result's own hardly.  Tolerance: that of
test_gpu_attn_prefix.py for queries that enter exactly, with the weights in two parts, each rounded by half a step:
U = 2^-16 (bf16) or 2^-22 (binary16, and n 2^-32 max |v| for those below its normal range)."""
import numpy as np
import pytest
import torch

import kv_share_ref as ref
from helpers import need_gpu
from test_gpu_attn_prefix import Case, STEP

pytestmark = pytest.mark.gpu


def _paired(wsw, q, cache, per, group, prefix=64, seed=0):
    c = Case(wsw, [(prefix, [prefix + 2 * i for i in range(per)])], kvh=1, group=group, q=q, cache=cache, seed=seed, junk=0.0)
    k, v = [x.view(-1, 1, c.d) for x in (c.kv.k, c.kv.v)]
    for r in range(per):
        even = c.slots(r, 0, c.lens[r])[::2].cuda()
        odd = c.slots(r, 0, c.lens[r])[1::2].cuda()
        v[odd] = -v[even]
        k[odd] = (k[even].float() * (1 + 2.0 ** -7)).to(k.dtype)
    c.vals = np.stack([x.double().cpu().numpy() for x in (k, v)])
    return c


@pytest.mark.parametrize("q,cache", [("bf16", "bf16"), ("fp16", "bf16"), ("fp16", "fp16"), ("bf16", "fp16")])
@pytest.mark.parametrize("per,group,wide", [(2, 4, False), (6, 8, False), (40, 8, False), (40, 8, True)])
def test_weights_in_two_parts(q, cache, per, group, wide):
    wsw = need_gpu()
    c = _paired(wsw, q, cache, per, group)
    if wide:  # room for rows so long that a unit has two row tiles
        narrow, width = c.table_d, 21 * 152 * 128 // (per * group // 128) // c.page + 9
        c.table_d = torch.full((per, width), -1, dtype=torch.int32, device="cuda")
        c.table_d[:, :narrow.shape[1]] = narrow
    half = cache == "bf16"
    for out, _ in (c.run(), c.run(share=False)):
        got, queries = out.double().cpu().numpy(), c.q.double().numpy()
        for r, n in enumerate(c.lens):
            p = np.arange(n)
            rows = c.table[r].numpy()[p // c.page] * c.page + p % c.page
            k, v = c.vals[0][rows], c.vals[1][rows]
            want, _, mag = ref.attend(queries[r], k, v, c.d ** -0.5)
            a = c.d ** -0.5 * float((np.abs(queries[r]) @ np.abs(k[:, 0]).T).max())
            parts = 2 if half and q == "fp16" else 1
            # fp16 over bf16: exact in two parts within a prefix, 2^-17 in the rest; bf16 over binary16: 2^-22
            e = a * ((0 if q == cache else 2.0 ** -17 if half else 2.0 ** -22) + (parts * c.d / 16 + 2) * 2.0 ** -23) + 2.0 ** -22
            sums = (2 * n / 16 + 32 + 160) * 2.0 ** -23
            lim = mag * (2 * e + (2.0 ** -16 if half else 2.0 ** -22) + sums) + n * 2.0 ** -32 * np.abs(v).max()
            bad = np.abs(got[r] - want) - (lim + STEP[q] * (np.abs(want) + lim) + 2.0 ** -25)
            assert (bad <= 0).all(), "request %d: over by %.3g of %.3g" % (r, bad.max(), lim.max())


@pytest.mark.parametrize("cache", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_of_positive_products(cache, d):
    """fp32 queries enter in two or three parts, the small ones first.  Sums of positive products grow evenly over the n = d / 16
    steps of the large part, to k / n of the score behind step k.  A step cuts its sum to fp32's bits (that it cuts half a
    last place in the mean does not hold: its addends are cut before they are added), so that it is off by less than a last
    place, 2^-23 of the sum so far: (1 + 2 + .. + n) / n = (n + 1) / 2 times 2^-23 of the score.  Were the small parts added
    behind, each of their n or 2 n steps would cut the whole score.  The lse's other roundings have either sign: their mean
    over 256 rows is below 2^-24."""
    wsw = need_gpu()
    c = Case(wsw, [(100, [100] * 32)], kvh=2, group=4, d=d, q="fp32", cache=cache, junk=0.0)
    c.q = c.q.abs() + 0.5
    k = c.kv.k.view(-1, 2, d)
    k.copy_(k.abs() + 0.5)
    vals = k.double().cpu().numpy()
    rows = c.table[0].numpy()[np.arange(100) // c.page] * c.page + np.arange(100) % c.page
    q = c.q.double().numpy().reshape(32, 2, 4, d)
    scale = 40.0 / float(np.einsum("rhgd,phd->rhgp", q, vals[rows]).mean())
    _, lse = c.run(scale)
    scale = float(np.float32(scale))
    x = np.einsum("rhgd,phd->rhgp", q, vals[rows]) * scale
    m = x.max(-1, keepdims=True)
    want = (m[..., 0] + np.log(np.exp(x - m).sum(-1))).reshape(32, 8)
    off = (lse.double().cpu().numpy() - want) / want
    assert abs(off.mean()) <= (d / 16 + 1) / 2 * 2.0 ** -23 + 2.0 ** -24, off.mean() * 2.0 ** 24
