"""Attention over shared prefixes under caps of every size: a score is off by parts of itself, not of the cap.

Tolerance: that of test_gpu_attn_prefix.py, but for softcap's tanh 32 2^-24 of the score: 24 2^-24 of the power's and the
reciprocal's form, and eight roundings of 2^-24 (cap, score and argument, or the series' sums and products)."""
import numpy as np
import pytest
import torch

import kv_share_ref as ref
from helpers import need_gpu
from test_gpu_attn_prefix import Case, STEP

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("softcap", [0.5, 7.0, 50.0, 1e3, 1e6, 1e10, 1e20, 1e35])
@pytest.mark.parametrize("q,cache", [("fp32", "fp16"), ("fp32", "bf16"), ("fp32", "q8_0"), ("fp16", "fp16"), ("bf16", "bf16")])
def test_caps_of_every_size(softcap, q, cache):
    wsw = need_gpu()
    c = Case(wsw, [(300, [300 + i for i in (0, 3, 40)])], kvh=2, group=4, q=q, cache=cache, qsigma=3.0, seed=7)
    scale, half, wide = c.d ** -0.5, cache == "bf16", q == "fp32"
    for share in (True, False):
        out, lse = c.run(scale, softcap=softcap, share=share)
        got, gl, queries = out.double().cpu().numpy(), lse.double().cpu().numpy(), c.q.double().numpy()
        for r, n in enumerate(c.lens):
            p = np.arange(n)
            rows = c.table[r].numpy()[p // c.page] * c.page + p % c.page
            k, v = c.vals[0][rows], c.vals[1][rows]
            want, wl, mag = ref.attend(queries[r], k, v, scale, softcap)
            heads = queries[r].reshape(c.kvh, c.group, -1)
            a = scale * max(float((np.abs(heads[h]) @ np.abs(k[:, h]).T).max()) for h in range(c.kvh))
            top = min(softcap, scale * max(float(np.abs(heads[h] @ k[:, h].T).max()) for h in range(c.kvh)))
            exact = q == cache or wide and half
            parts = 3 if wide and half else 2 if wide else 1
            e = a * ((0 if exact else 2.0 ** -22) + (parts * c.d / 16 + 2) * 2.0 ** -23) + 32 * 2.0 ** -24 * top + 2.0 ** -22
            u = (0 if half else 2.0 ** -22) if wide else 2.0 ** -16 if half else 2.0 ** -22
            sums = (3 * n / 16 + 32 + 160) * 2.0 ** -23
            lim = mag * (2 * e + u + sums) + n * 2.0 ** -32 * np.abs(v).max()
            bad = np.abs(got[r] - want) - (lim + STEP[q] * (np.abs(want) + lim) + 2.0 ** -25)
            assert (bad <= 0).all(), "request %d: over by %.3g of %.3g" % (r, bad.max(), lim.max())
            lim = e + 2.0 ** -22 + sums + 2.0 ** -22 * np.abs(wl)
            assert (np.abs(gl[r] - wl) <= lim).all(), "request %d: lse off by %.3g" % (r, np.abs(gl[r] - wl).max())


def test_a_cap_far_above_the_scores_changes_nothing():
    """Caps from 1e4 times the scores on bend them by less than 1e-8: the result without one."""
    wsw = need_gpu()
    c = Case(wsw, [(500, [500 + i for i in (1, 30)])], kvh=2, group=4, q="fp32", cache="fp16", qsigma=3.0)
    want, want_lse = c.run(0.1)
    for softcap in (1e6, 1e8, 1e12):
        out, lse = c.run(0.1, softcap=softcap)
        assert float((out - want).abs().max()) < 2e-4 and float((lse - want_lse).abs().max()) < 1e-4


@pytest.mark.parametrize("softcap", [1e-30, 1e-37, 5e-38, 1e-39, 1e-44])
@pytest.mark.parametrize("q,cache", [("fp32", "fp16"), ("bf16", "bf16"), ("bf16", "q8_0")])
def test_caps_below_every_score(softcap, q, cache):
    """Every score is +-softcap, next to nothing, or 0: the values' mean, for queries of zeros, too."""
    wsw = need_gpu()
    c = Case(wsw, [(300, [300 + i for i in (0, 3, 40)])], kvh=2, group=4, q=q, cache=cache, seed=7)
    c.q[1] = 0
    c.q[2, 3] = 0
    for scale in (0.1, -3.0):
        for share in (True, False):
            out, lse = c.run(scale, softcap=softcap, share=share)
            for r, n in enumerate(c.lens):
                p = np.arange(n)
                rows = c.table[r].numpy()[p // c.page] * c.page + p % c.page
                want = np.repeat(c.vals[1][rows].mean(0), c.group, 0)
                mag = np.abs(c.vals[1][rows]).mean(0).max()
                # weights and their sums: (300 / 16 + 192) 2^-23 and 2^-16 for the parts; then the result's rounding
                lim = mag * (211 * 2.0 ** -23 + 2.0 ** -16) + n * 2.0 ** -32 * mag
                assert (np.abs(out[r].double().cpu().numpy() - want) <= lim + STEP[q] * (np.abs(want) + lim)).all(), r
                assert (np.abs(lse[r].double().cpu().numpy() - np.log(n)) <= 211 * 2.0 ** -23 + 2.0 ** -22 * 6).all(), r
