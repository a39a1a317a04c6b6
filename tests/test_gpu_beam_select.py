"""Beam selection on the GPU against the definition in 64 bits.

A candidate's score is off by the error of its row's lse.  A term exp((x - m) scale) = 2^t has its exponent
rounded three times (difference, product, scale log2 e), 3 2^-24 |t|, and is within 2^-22 of the power: the sum is off by
2^-22 + 3 2^-24 ln 2 times the mean of |t| over the distribution, which is below its entropy, log2(vocab) <= 18:
2^-18.7.  A thread adds at most 16 pairs a tile, three tiles here: 51 2^-24 = 2^-18.3 (above, 64 bits).  Together
E = 2^-17.  The ids are asked for where no two scores that decide lie within 2 E of each other (equal ones
apart: they rank by index); elsewhere the scores alone."""
import math

import numpy as np
import pytest
import torch

import kv_share_ref as ref
from helpers import need_gpu

pytestmark = pytest.mark.gpu

E = 2.0 ** -17
T = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def _check(wsw, x, scores, ends=(), scale=1.0, ws=None, opts=None):
    """x [requests][beams][vocab] on the device, scores numpy [requests][beams]."""
    n, beams, vocab = x.shape
    s = torch.tensor(scores, dtype=torch.float32, device="cuda")
    logits = x.view(n * beams, vocab) if x.is_contiguous() else x[0]
    r = wsw.beam_select(logits, s, ends, scale=scale, ws=ws, opts=opts)
    host = x.double().cpu().numpy()
    got = [t.cpu().numpy() for t in r]
    decided = 0
    for q in range(n):
        nxt, ended, order = ref.beam(host[q], s[q].double().cpu().numpy(), set(ends), scale)
        near = np.isfinite(order[:-1]) & np.isfinite(order[1:]) & (np.diff(order) > -2 * E) & (np.diff(order) != 0)
        for want, (parent, token, score) in ((nxt, got[:3]), (ended, got[3:])):
            k = len(want)
            assert (parent[q, k:] == -1).all() and (token[q, k:] == -1).all() and (score[q, k:] == -np.inf).all()
            assert (parent[q, :k] >= 0).all()
            if near.any():
                continue
            decided += 1
            assert parent[q, :k].tolist() == [q * beams + c[0] for c in want]
            assert token[q, :k].tolist() == [c[1] for c in want]
        for want, score in ((nxt, got[2]), (ended, got[5])):
            for i, c in enumerate(want):
                if not near.any() or want is nxt and not ends:
                    assert abs(float(score[q, i]) - c[2]) <= E + 2.0 ** -24 * (abs(c[2]) + E)
    return r, decided


def _logits(seed, n, beams, vocab, kind="fp32", spread=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, 1, vocab, generator=g, device="cuda") * spread + torch.randn(n, beams, vocab, generator=g, device="cuda")
    return x.to(T[kind])


def _scores(seed, n, beams):
    g = np.random.default_rng(seed)
    return (-np.cumsum(g.random((n, beams)) * 2, 1)).astype(np.float32)


@pytest.mark.parametrize("n,beams,vocab", [(1, 1, 1), (1, 4, 3), (2, 3, 33), (1, 4, 5000), (3, 5, 4097), (5, 16, 1001),
                                           (1, 32, 9000), (40, 8, 2050), (1, 2, 152064), (700, 1, 129), (64, 4, 20011)])
@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("ends", [0, 1, 3])
def test_matches_the_definition(n, beams, vocab, kind, ends):
    wsw = need_gpu()
    if beams * (1 + ends) > 32:
        ends = 0
    x = _logits(n + beams + vocab, n, beams, vocab, kind)
    tokens = [0, vocab - 1, vocab // 2][:ends]
    for t in tokens:
        x[:, ::2, t] = 9.0
    _, decided = _check(wsw, x, _scores(vocab, n, beams), tokens)
    assert decided > 0 or kind != "fp32" or vocab < 10


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_scale_and_row_strides(kind):
    wsw = need_gpu()
    g = torch.Generator(device="cuda").manual_seed(1)
    room = torch.randn(6, 3001, generator=g, device="cuda").to(T[kind]) * 2
    for off, vocab in ((0, 2999), (1, 3000), (3, 2000)):
        x = room[:, off: off + vocab].unsqueeze(0)
        for scale in (0.5, 1.0, 3.0):
            _check(wsw, x, _scores(off, 1, 6), [7], scale=scale)


def test_forbidden_tokens_dead_beams_and_rows_without_candidates():
    wsw = need_gpu()
    x = _logits(5, 6, 4, 700)
    s = _scores(6, 6, 4)
    x[0, :, 3:] = -math.inf            # three tokens a beam are left: 12 candidates
    s[0, 1:] = -math.inf               # ... and one beam: the first step, three candidates
    x[1, 0] = -math.inf                # a row of nothing
    x[2, 1, 5], x[2, 2, 699] = math.nan, math.inf
    s[3] = -math.inf                   # no beam at all
    s[4, 0], s[4, 1] = math.nan, math.inf
    x[5] = torch.finfo(torch.float32).min  # the type's lowest value: an even distribution
    s[5] = [-3, -1, -2, -1]
    r, _ = _check(wsw, x, s, [2])
    assert (r.parent[3] == -1).all() and (r.score[3] == -math.inf).all()
    assert r.parent[0].tolist()[2:] == [-1, -1] and r.end_token[0].tolist()[0] == 2  # token 2 ends
    assert set(r.parent[1].tolist()) <= {5, 6, 7} and set(r.parent[2].tolist()) <= {8, 11}
    # beams 1 and 3 of the last request tie throughout: beam 1's tokens, from the lowest
    assert r.parent[5].tolist() == [21] * 4 and r.token[5].tolist() == [0, 1, 3, 4]


@pytest.mark.parametrize("vocab", [1000, 20001, 152064])
@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
def test_copies_of_a_beam_tie_and_rank_by_index(vocab, kind):
    """Equal rows at different alignments (vocab odd): the sums differ in their order only."""
    wsw = need_gpu()
    x = _logits(vocab, 2, 1, vocab, kind).expand(2, 4, vocab).contiguous()
    s = np.full((2, 4), -2.5, np.float32)
    r, _ = _check(wsw, x, s)
    for q in range(2):
        best = int(x[q, 0].float().argmax())
        assert r.parent[q].tolist() == [4 * q + b for b in range(4)]
        assert all(float(x[q, 0, t]) == float(x[q, 0, best]) for t in r.token[q].tolist())
        assert len(set(r.score[q].tolist())) == 1


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("order", ["rising", "falling", "equal", "raised tenth"])
def test_uneven_rows(kind, order):
    wsw = need_gpu()
    x = _logits(9, 2, 3, 30000, "fp32")
    if order == "rising":
        x = x.sort(-1).values
    elif order == "falling":
        x = x.sort(-1, descending=True).values
    elif order == "equal":
        x = torch.zeros_like(x) + torch.arange(3, device="cuda").view(1, 3, 1)
    else:
        x[..., 20000:23000] += 6
    _check(wsw, x.to(T[kind]).contiguous(), _scores(2, 2, 3), [29999])


def test_one_workspace_serves_calls_of_different_sizes():
    wsw = need_gpu()
    sizes = [(1, 4, 152064), (300, 1, 5000), (50, 10, 700), (1, 1, 9), (9, 8, 40000)]
    ws = torch.zeros(max(wsw.beam_select_workspace_bytes(*s, 1) for s in sizes), dtype=torch.uint8, device="cuda")
    for turn in range(2):
        for i, (n, beams, vocab) in enumerate(sizes):
            _check(wsw, _logits(i + turn, n, beams, vocab), _scores(i, n, beams), [1], ws=ws, opts={"pdl": turn})
    assert (ws[:4 * 16384] == 0).all()


def test_results_are_the_same_in_a_graph_and_on_another_stream():
    wsw = need_gpu()
    x, s = _logits(3, 7, 5, 30011).view(35, 30011), torch.tensor(_scores(3, 7, 5), device="cuda")
    ws = torch.zeros(wsw.beam_select_workspace_bytes(7, 5, 30011, 1), dtype=torch.uint8, device="cuda")
    want = wsw.beam_select(x, s, [4], ws=ws)
    out = wsw.beam_select_out(7, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        wsw.beam_select(x, s, [4], ws=ws, out=out)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    for t in out:
        t.fill_(7)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wsw.beam_select(x, s, [4], ws=ws, out=out)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_two_streams_at_once():
    """Each call with its own workspace: the results of calls alone."""
    wsw = need_gpu()
    g = torch.Generator(device="cuda").manual_seed(0)
    jobs = []
    for n in (3, 70):
        x, s = torch.randn(n * 4, 60000, generator=g, device="cuda") * 2, torch.zeros(n, 4, device="cuda")
        want = [t.clone() for t in wsw.beam_select(x, s, [5])]
        ws = torch.zeros(wsw.beam_select_workspace_bytes(n, 4, 60000, 1), dtype=torch.uint8, device="cuda")
        jobs.append((x, s, want, ws, wsw.beam_select_out(n, 4), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(30):
        for x, s, _, ws, out, stream in jobs:
            with torch.cuda.stream(stream):
                wsw.beam_select(x, s, [5], out=out, ws=ws)
    torch.cuda.synchronize()
    for _, _, want, _, out, _ in jobs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("vocab", [40, 30011])
@pytest.mark.parametrize("beams,ends", [(1, 8), (2, 8), (4, 7), (8, 3), (10, 2), (16, 1)])
def test_end_tokens_lead_every_row(vocab, beams, ends):
    """The end tokens are each row's largest: all places of a request's first candidates may be theirs."""
    wsw = need_gpu()
    x = _logits(beams, 5, beams, vocab)
    tokens = [(7 * i + 3) % vocab for i in range(ends)]
    x[:3, :, tokens] += 15
    x[3, :beams // 2 + 1, tokens] += 15
    decided = _check(wsw, x, _scores(0, 5, beams), tokens)[1]
    decided += _check(wsw, x, np.zeros((5, beams)), tokens + [vocab + 5] if ends < 8 and beams * (2 + ends) <= 32 else tokens)[1]
    assert decided >= 2
