"""Paged decode attention over lists of tiles so long that a pair counts extra (4 * 152 tiles for each
warp of a CTA), for the shapes whose cuts differ: head_dim 256 (four warps, where a cut can stay within a
pair's extra places), 16 query rows, several passes over a pair, and third parts of q."""
import numpy as np
import pytest

from helpers import need_gpu
from test_gpu_attn_paged import Case

pytestmark = pytest.mark.gpu


def _offsets(lens, tile, pairs, warps):
    """How far into a long pair (more than 512 positions) the 152 cuts fall, in places of the list; empty
    if the list is too short for extra counts."""
    tiles = [-(-n // tile) for n in lens]
    if sum(tiles) * pairs < 4 * 152 * warps:
        return set()
    counted = [(t + 4 if t else 0, t) for t in tiles for _ in range(pairs)]
    run = -(-sum(c for c, _ in counted) // 152)
    begins = np.cumsum([0] + [c for c, _ in counted])
    at = set()
    for s in range(run, int(begins[-1]), run):
        i = int(np.searchsorted(begins, s, side="right")) - 1
        if counted[i][1] > 512 // tile:
            at.add(s - int(begins[i]))
    return at


@pytest.mark.parametrize("d,group,cache,q,kvh,tile,warps,passes,longest", [
    (256, 4, "fp16", "fp32", 2, 16, 4, 1, 1100),
    (256, 10, "bf16", "bf16", 2, 16, 4, 1, 1100),
    (256, 8, "q8_0", "fp32", 2, 16, 4, 1, 1100),
    (256, 3, "bf16", "fp32", 2, 16, 4, 1, 1100),
    (256, 20, "fp16", "fp16", 1, 16, 4, 2, 1100),
    (128, 10, "bf16", "bf16", 4, 16, 8, 1, 1500),
    (128, 40, "fp16", "fp32", 1, 16, 8, 3, 2500),
    (128, 12, "q8_0", "bf16", 4, 32, 8, 1, 3000),
    (128, 9, "bf16", "fp32", 4, 16, 8, 1, 1500),
    (64, 16, "fp16", "fp16", 4, 16, 8, 1, 1500),
    (64, 7, "q8_0", "fp32", 4, 32, 12, 1, 4500)])
def test_lists_with_cuts_at_every_place_of_a_pair(d, group, cache, q, kvh, tile, warps, passes, longest):
    wsw = need_gpu()
    done = 0
    for seed in range(200):
        g = np.random.default_rng(seed)
        lens = [int(x) for x in g.integers(520, longest, 40)] + [int(x) for x in g.integers(0, 300, 6)] + [0]
        g.shuffle(lens)
        if set(range(5)) <= _offsets(lens, tile, kvh * passes, warps):
            Case(wsw, lens, kvh=kvh, group=group, d=d, cache=cache, q=q, page=[16, 64, 8][seed % 3], nhd=seed % 2 == 0,
                 seed=seed).check()
            done += 1
        if done == 2:
            return
    raise AssertionError("no such lists")
