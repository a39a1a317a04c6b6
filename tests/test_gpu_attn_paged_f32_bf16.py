"""fp32 queries over bf16 pages: scores, softmax weights and outputs carry fp32, against the formula
in 64 bits.  The inputs leave one product in each score and in each output, so that the bounds are a
few roundings (u = 2^-24) and what bf16 parts might drop shows."""
import math

import numpy as np
import pytest
import torch

from helpers import need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _pages(wsw, rows):
    """A cache of bf16 pages of 16 from [positions][heads][dim] rows, one request's, in order."""
    n, h, d = rows[0].shape
    kv = [torch.cat([x, x.new_zeros(-n % 16, h, d)]).view(-1, 16, h, d).to(torch.bfloat16).cuda() for x in rows]
    table = torch.arange(kv[0].shape[0], dtype=torch.int32, device="cuda")[None]
    return wsw.PagedKV(*kv), table, torch.tensor([n], dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 8, 13, 40])
def test_scores_carry_fp32(d, group):
    """One position: lse is its score.  Roundings: scale log2 e (2), the product (1), the sum and
    difference with the weights' shift (2, of |x| + 8 ln 2), ln 2 and its product (2)."""
    wsw = need_gpu()
    g = torch.Generator().manual_seed(d + group)
    q = torch.zeros(1, 2 * group, d)
    at = torch.randint(0, d, (2 * group,), generator=g)
    q[0, torch.arange(2 * group), at] = torch.randn(2 * group, generator=g) * 40
    k = (torch.randn(1, 2, d, generator=g) + 2).to(torch.bfloat16)
    kv, table, lens = _pages(wsw, [k.float(), torch.zeros(1, 2, d)])
    lse = torch.empty(1, 2 * group, device="cuda")
    wsw.attn_paged_decode(q.cuda(), kv, table, lens, scale=0.7, lse=lse)
    x = 0.7 * (q[0].double().view(2, group, d) * k[0].double()[:, None]).sum(-1).numpy().ravel()
    off = np.abs(lse[0].double().cpu().numpy() - x)
    assert (off <= 8 * U * (np.abs(x) + 8 * math.log(2))).all(), (off / U / (np.abs(x) + 8 * math.log(2))).max()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 8, 13])
def test_weights_carry_fp32(d, group):
    """16 positions of scores within 1/2 and values that are the identity: an output is one weight over
    their sum.  A weight: the score's 4 u of 1/2, the exponential's 4 u; an output: that twice (its own
    and the sum's), 6 u for three products' sums, 6 u for the sum of weights, 3 u for the quotient."""
    wsw = need_gpu()
    g = torch.Generator().manual_seed(d * group)
    q = torch.zeros(1, group, d)
    q[0, :, 0] = torch.rand(group, generator=g) - 0.5
    k = torch.zeros(16, 1, d)
    k[:, 0, 0] = torch.rand(16, generator=g) * 2 - 1
    k = k.to(torch.bfloat16)
    v = torch.zeros(16, 1, d)
    v[torch.arange(16), 0, torch.arange(16) * (d // 16)] = 1.0
    kv, table, lens = _pages(wsw, [k.float(), v])
    out = wsw.attn_paged_decode(q.cuda(), kv, table, lens, scale=1.0)
    w = np.exp(q[0, :, :1].double().numpy() * k[:, 0, 0].double().numpy())
    want = w / w.sum(-1, keepdims=True)
    off = np.abs(out[0, :, :: d // 16].double().cpu().numpy() / want - 1)
    assert off.max() <= (2 * (4 * 0.5 + 4) + 6 + 6 + 3) * U, off.max() / U
