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
