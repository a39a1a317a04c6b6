"""The operators of a beam step together, as examples/beam_search.py runs them: every stage of
replayed steps against its definition on the tensors that the step found and left, and every
beam's keys and values after many forks against those that its lineage wrote."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

import kv_share_ref as ref
from helpers import need_gpu

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "beam_search.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("beam_search", _PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _np(t):
    return t.cpu().numpy().copy()


def _rows(b, r, n, layer=0):
    """What row r's first n positions hold: K and V (codes and scales, too) as bytes."""
    kv = b.caches[layer]
    p = torch.arange(n, device="cuda")
    page, off = b.table[r].long()[p // b.page_size], p % b.page_size
    return [x[page, off].contiguous().view(torch.uint8).cpu().numpy() for x in (kv.k, kv.v, kv.kd, kv.vd) if x is not None]


@pytest.mark.parametrize("cache", ["fp16", "bf16", "q8_0"])
@pytest.mark.parametrize("share", [False, True])
def test_replayed_steps_match_the_definitions(example, cache, share):
    need_gpu()
    page, beams, steps = 4, 3, 14
    model = example.Decoder(layers=2, vocab=300)
    prompts = [[5, 6, 7, 8, 9], [1], list(range(20, 43))]
    b = example.Beams(model, prompts, beams, end_token=3, page_size=page, max_new=steps + 1, cache=cache, share=share)
    n, pool = b.n, b.pages
    assert b.lens.tolist() == [len(p) - 1 for p in prompts for _ in range(beams)]
    kept = [_rows(b, r, int(b.lens[r])) for r in range(n)]
    for step in range(steps):
        table, lens, scores, head = _np(b.table), _np(b.lens), _np(b.scores), int(b.head)
        free = _np(b.free)
        assert free[head:].tolist() == ref.compact(lens, table, page, pool)[1]
        b.step()
        # the plan: a fresh page for rows whose last one was full, in row order
        taken = 0
        for r in range(n):
            if lens[r] % page == 0:
                table[r, lens[r] // page] = free[head + taken]
                taken += 1
        lens = lens + 1
        # selection from the step's logits
        logits = _np(b.logits.double())
        parent, token = _np(b.chosen.parent), _np(b.chosen.token)
        for q in range(len(prompts)):
            nxt, ended, order = ref.beam(logits[q * beams:(q + 1) * beams], scores[q].astype(np.float64), {3})
            gaps = np.diff(order[np.isfinite(order)])
            if not ((gaps > -2.0 ** -16) & (gaps != 0)).any():
                k = len(nxt)
                assert parent[q, :k].tolist() == [q * beams + c[0] for c in nxt] and (parent[q, k:] == -1).all()
                assert token[q, :k].tolist() == [c[1] for c in nxt]
                assert b.chosen.end_token[q, :len(ended)].tolist() == [3] * len(ended)
        # the children's rows, the copies and the free list
        want = ref.fork(parent.ravel(), lens, free, head + taken, table, page, table)
        assert np.array_equal(_np(b.table), want[0]) and b.lens.tolist() == want[1].tolist()
        assert int(b.fork.copies.count) == len(want[3])
        after = ref.compact(want[1], want[0], page, pool)
        assert int(b.head) == after[2] and _np(b.free)[after[2]:].tolist() == after[1]
        # every beam's positions are those of its lineage
        now = []
        for i, p in enumerate(parent.ravel()):
            got = _rows(b, i, int(b.lens[i]))
            if p >= 0:
                assert all(np.array_equal(x[:-1], y) for x, y in zip(got, kept[p])), (step, i)
            now.append(got)
        kept = now
    assert int(b.err) == 0


@pytest.mark.parametrize("cache", ["fp16", "bf16", "q8_0"])
def test_shared_and_single_attention_agree_on_a_step(example, cache):
    """The step's attention over the forked rows: once for the prefix against row by row."""
    wsw = need_gpu()
    model = example.Decoder(layers=1, vocab=200)
    b = example.Beams(model, [list(range(50)), [7] * 9], 4, page_size=8, max_new=9, cache=cache)
    for _ in range(5):
        b.step()
    g = torch.Generator(device="cuda").manual_seed(0)
    q = torch.randn(b.n, model.q_heads, model.head_dim, generator=g, device="cuda")
    one = wsw.attn_paged_decode(q, b.caches[0], b.table, b.lens)
    both = wsw.attn_paged_prefix(q, b.caches[0], b.table, b.lens, b.groups, b.prefix, share=True)
    # fp32 queries: both are within 2^-17 of sums of |score| some 40, of values below 5
    assert (one - both).abs().max() <= 2 * 2.0 ** -17 * 40 * 5


def test_search_returns_hypotheses(example):
    need_gpu()
    model = example.Decoder(layers=1, vocab=120)
    found, b = example.search(model, [[5, 6, 7], [9] * 20], 10, beams=4, end_token=1, page_size=8)
    for hypotheses in found:
        assert len(hypotheses) >= 4
        for tokens, score in hypotheses:
            assert 1 <= len(tokens) <= 10 and score < 0 and math.isfinite(score)
            assert 1 not in tokens[:-1]
