"""Beam selection over rows that are copies, or nearly: equal rows tie and rank by index, others rank by what sets them
apart.  Two allowed tokens t nats apart leave ln S = ln(1 + e^-t), 8.3e-7 for 14 and 3.1e-7 for 15; the sum is off by
2^-23 at most (one rounding of 1 + e^-t), 1.2e-7, and by 2^-22 of e^-t."""
import math

import numpy as np
import pytest
import torch

from helpers import need_gpu
from test_gpu_beam_select import T, _check, _logits, _scores

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("vocab", [16, 1001, 50021, 152064])
@pytest.mark.parametrize("apart", [(14, 15), (15, 14), (14, 15, 14, 16), (13, 14, 15, 13, 16, 14)])
def test_near_copies_rank_by_their_sums(kind, vocab, apart):
    wsw = need_gpu()
    for top, other in ((3, 4), (vocab - 1, 0), (0, vocab - 1), (vocab // 2, 7)):
        x = torch.full((1, len(apart), vocab), -math.inf, dtype=T[kind], device="cuda")
        for b, t in enumerate(apart):
            x[0, b, top], x[0, b, other] = 20, 20 - t
        r = wsw.beam_select(x[0], torch.full((1, len(apart)), -1.0, device="cuda"))
        want = sorted(range(len(apart)), key=lambda b: (-apart[b], b))  # the larger distance, the smaller sum
        assert r.parent[0].tolist() == want and r.token[0].tolist() == [top] * len(apart)


@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("vocab", [7, 129, 4099, 50021, 100003])
def test_copies_tie_at_every_alignment(kind, vocab):
    """Rows of an odd length begin at every place within 16 bytes, views one element on, too."""
    wsw = need_gpu()
    row = _logits(vocab, 1, 1, vocab, kind)[0, 0]
    room = torch.zeros(9 * vocab + 1, dtype=T[kind], device="cuda")
    for start in (0, 1):
        x = room[start: start + 9 * vocab].view(9, vocab)
        x[:] = row
        x[4] = row.flip(0)
        r = wsw.beam_select(x, torch.full((1, 9), -2.0, device="cuda"))
        best = torch.sort(row.float(), descending=True, stable=True)
        score = {b: [float(s) for p, s in zip(r.parent[0].tolist(), r.score[0].tolist()) if p == b] for b in range(9)}
        assert [p for p in r.parent[0].tolist() if p != 4] == [b for b in range(9) if b != 4][:9 - len(score[4])]
        assert len({s for b in range(9) if b != 4 for s in score[b]}) == 1
        assert all(float(row[t]) == float(best.values[0]) for p, t in zip(r.parent[0].tolist(), r.token[0].tolist()) if p != 4)


@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("order", ["rising", "falling", "equal", "raised tenth"])
def test_uneven_rows_at_every_alignment(kind, order):
    wsw = need_gpu()
    vocab = 30001
    x = _logits(9, 1, 9, vocab, "fp32")
    if order == "rising":
        x = x.sort(-1).values
    elif order == "falling":
        x = x.sort(-1, descending=True).values
    elif order == "equal":
        x = torch.zeros_like(x) + torch.arange(9, device="cuda").view(1, 9, 1)
    else:
        x[..., 20000:23000] += 6
    _check(wsw, x.to(T[kind]).contiguous(), _scores(2, 1, 9), [vocab - 1])


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_masks_of_the_lowest_value(kind):
    """Tokens masked by the type's lowest value are candidates behind all others while their scores are finite in fp32, by
    the lower token; a scale above 1 takes them out of fp32's range: none."""
    wsw = need_gpu()
    low = torch.finfo(T[kind]).min
    x = torch.full((6, 5000), low, dtype=T[kind], device="cuda")
    x[:, 4000], x[:, 17] = 3, 1
    s = torch.tensor([[-1.0, -2, -3], [-1.0, -1, -1]], device="cuda")
    r = wsw.beam_select(x[:3, :600], s[:1])  # one token of each row is allowed
    assert r.parent.tolist() == [[0, 1, 2]] and r.token.tolist() == [[17] * 3] and r.score.tolist() == [[-1, -2, -3]]
    one = x.clone()
    one[1:3], one[4:] = low, low
    s[0, 1:] = -math.inf
    r = wsw.beam_select(one, s)
    assert r.token[0].tolist() == [4000, 17, 0] and float(r.score[0, 2]) < -3e38 and r.parent[0].tolist() == [0] * 3
    # rows of nothing else are even: ln 5000 below their scores
    assert r.parent[1].tolist() == [3, 3, 4] and r.token[1].tolist() == [4000, 17, 0]
    assert abs(float(r.score[1, 2]) + 1 + math.log(5000)) < 1e-5
    r = wsw.beam_select(one, s, scale=2.0)
    assert r.token[0].tolist() == [4000, 17, -1] and r.parent[0].tolist() == [0, 0, -1] and float(r.score[0, 2]) == -math.inf
    assert r.parent[1].tolist() == [3, 3, 4] and r.token[1].tolist() == [4000, 17, 0]
