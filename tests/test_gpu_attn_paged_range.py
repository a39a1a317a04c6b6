"""Paged decode attention at the ends of its types' ranges, against the formula in 64 bits (the
inputs, bounds and check of test_gpu_attn_paged)."""
import numpy as np
import pytest
import torch

import kv_step_ref as ref
from helpers import need_gpu
from test_gpu_attn_paged import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,group,q", [(128, 4, "bf16"), (64, 10, "fp32"), (256, 1, "bf16"), (128, 16, "bf16")])
def test_bf16_values_near_the_largest(d, group, q):
    """Values up to 2^125: a weighted sum of them overflows only where weights grow past 1."""
    wsw = need_gpu()
    c = Case(wsw, [1, 2, 40, 300], group=group, d=d, q=q, cache="bf16")
    c.kv.v.copy_(c.kv.v.double() * 2.0 ** 122)
    c.vals[1] *= 2.0 ** 122
    c.check()


@pytest.mark.parametrize("cache,page", [("fp16", 8), ("q8_0", 16)])
def test_the_last_positions_that_there_can_be(cache, page):
    """Lengths just below 2^31 - 4096.  The window keeps the work small; the block table is as long
    as the length."""
    wsw = need_gpu()
    pages = ((1 << 31) - 4096) // page
    length, window, kvh, group, d = pages * page - 3, 100, 2, 4, 128
    table = torch.arange(pages, dtype=torch.int32, device="cuda").remainder_(3)[None]
    c = Case(wsw, [3 * page], kvh=kvh, group=group, cache=cache, page=page, extra=0, seed=page)
    c.lens_d.fill_(length)
    c.table_d = table
    out, lse = c.run(window=window)
    p = np.arange(length - window, length)
    rows = p // page % 3 * page + p % page
    want, wl, mag, terms = ref.attend(c.q[0].double().numpy(), c.vals[0][rows], c.vals[1][rows], d ** -0.5)
    # test_gpu_attn_paged's bounds, with its bf16 terms
    e = terms * (2.0 ** -17 + (d / 16 + 2) * 2.0 ** -23) + 2.0 ** -22
    lim = mag * (2 * e + 2.0 ** -17 + 8 * 2.0 ** -23) + 2.0 ** -24 * np.abs(want) + 2.0 ** -25
    assert (np.abs(out[0].double().cpu().numpy() - want) <= lim).all()
    lim = e + 2.0 ** -22 + 8 * 2.0 ** -23 + 2.0 ** -22 * np.abs(wl)
    assert (np.abs(lse[0].double().cpu().numpy() - wl) <= lim).all()


@pytest.mark.parametrize("cache,q", [("fp16", "fp32"), ("bf16", "fp32"), ("bf16", "bf16"), ("q8_0", "fp16")])
@pytest.mark.parametrize("softcap", [1e38, 3e38])
def test_a_cap_near_the_largest_number_is_none(cache, q, softcap):
    wsw = need_gpu()
    c = Case(wsw, [1, 40, 300], cache=cache, q=q)
    for got, want in zip(c.run(softcap=softcap), c.run()):
        assert torch.equal(got, want)
