"""The operators of a decode step together, as examples/paged_decode.py runs them: every
stage of a replayed step against its definition on the tensors that the step left."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

import kv_step_ref as ref
from helpers import need_gpu

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_decode.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("paged_decode", _PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _np(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("cache", ["fp16", "bf16", "q8_0"])
def test_a_replayed_step_matches_the_definitions(example, cache):
    wsw = need_gpu()
    model = example.Decoder(layers=2, vocab=1000)
    prompts = [[1], [5, 6, 7], list(range(40)), [9] * 17, [3, 2]]
    steps = 6
    out, logprob, s = example.generate(model, prompts, steps, cache)
    longest = max(len(p) for p in prompts) + steps
    fed = longest - 1  # every request took a token per step
    assert all(len(o) >= len(p) + steps for o, p in zip(out, prompts))
    assert s.lens.tolist() == [fed] * 5
    # the plan: every request's own pages, in the order in which they were opened
    per = -(-fed // 16)
    table = s.table.cpu().numpy()
    used = table[:, :per]
    assert len(set(used.ravel().tolist())) == 5 * per and used.min() >= 0 and (table[:, per:] == -1).all()
    assert int(s.first_free) == 5 * per
    slots = used[:, (fed - 1) // 16] * 16 + (fed - 1) % 16
    assert np.array_equal(s.plan.slots.cpu().numpy(), slots) and (s.plan.positions.cpu().numpy() == fed - 1).all()
    # the last layer's attention over the cache that the steps wrote
    kv = s.caches[-1]
    if cache == "q8_0":
        k, v = (wsw.dequant_q8_0_kv(x.view(-1, 2, 128), d.view(-1, 2, 4)).permute(1, 0, 2) for x, d in
                ((kv.k, kv.kd), (kv.v, kv.vd)))
    else:
        k, v = kv.k.view(-1, 2, 128), kv.v.view(-1, 2, 128)
    k, v, q, got = _np(k), _np(v), _np(s.q[-1]), _np(s.attn[-1])
    p = np.arange(fed)
    for r in range(5):
        rows = used[r, p // 16] * 16 + p % 16
        want, _, mag, terms = ref.attend(q[r], k[rows], v[rows], 1 / math.sqrt(128))
        # as the attention's own tests derive it (fp32 q over 16-bit rows)
        e = terms * ((2.0 ** -17 if cache == "bf16" else 2.0 ** -22) + 10 * 2.0 ** -23) + 2.0 ** -22
        lim = mag * (2 * e + (2.0 ** -17 if cache == "bf16" else 2.0 ** -22) + (fed / 16 + 1) * 2.0 ** -23)
        assert (np.abs(got[r] - want) <= lim + 2.0 ** -24 * (np.abs(want) + lim)).all(), r
    # the rotated q of the last step, from the QKV rows that it left
    f, m = ref.rope_freqs(128, scaling="by_parts", factor=4.0, original=32768)
    raw = _np(s.qkv[:, :8])
    yq = ref.rotate(raw, np.full(5, fed - 1), f, m, False)
    mag = np.concatenate([np.abs(raw[..., :64]) + np.abs(raw[..., 64:])] * 2, -1) * m
    assert (np.abs(q - yq) <= 11 * 2.0 ** -24 * mag + 2.0 ** -24 * (np.abs(yq) + 11 * 2.0 ** -24 * mag)).all()
    # the report on the logits
    logits = _np(s.logits)
    for r in range(5):
        _, _, lse, ent, order, best, _ = ref.logprobs(logits[r], 0, 1.0, 4)
        assert s.report.top_id[r].tolist() == order.tolist()
        # 1000 logits: sums within 2^-21 + 24 2^-24, a few roundings of the value
        assert np.allclose(_np(s.report.top_logprob[r]), best, rtol=2.0 ** -22, atol=2.0 ** -18)
        assert abs(float(s.report.lse[r]) - lse) <= 2.0 ** -18 + 2.0 ** -22 * abs(lse)


def test_replay_equals_the_uncaptured_step(example):
    """The same tokens fed to a server that never captures give the same bits."""
    need_gpu()
    model = example.Decoder(layers=1, vocab=500)
    servers = [example.Server(model, 3, pages=12) for _ in range(2)]
    for t in range(20):
        for s in servers:
            s.tokens.copy_(torch.tensor([t, 2 * t, 499 - t], dtype=torch.int32))
        servers[0].step()
        servers[1]._step()
        assert torch.equal(servers[0].report.top_id, servers[1].report.top_id), t
        assert torch.equal(servers[0].report.lse, servers[1].report.lse), t
    assert torch.equal(servers[0].table, servers[1].table)


def test_a_server_out_of_pages_reports_it(example):
    need_gpu()
    model = example.Decoder(layers=1, vocab=500)
    s = example.Server(model, 3, pages=2)
    s.step()
    assert int(s.err) == 8  # the third request got no page
    assert s.lens.tolist() == [1, 1, 0] and s.plan.slots.tolist()[2] == -1
    assert (s.attn[0][2] == 0).all()


@pytest.mark.parametrize("cache,pages", [("fp16", 17000), ("q8_0", 33500)])
def test_a_cache_whose_offsets_pass_32_bits(cache, pages):
    """Rows written and read past 2^32 bytes (and 2^31 elements) of each buffer equal those of a small cache."""
    wsw = need_gpu()
    page, h, d, n, length = 256, 4, 128, 3, 300
    g = torch.Generator().manual_seed(3)
    code = torch.int8 if cache == "q8_0" else torch.float16

    def make(count):
        kv = [torch.empty((count, page, h, d), dtype=code, device="cuda") for _ in range(2)]
        sc = [torch.empty((count, page, h, d // 32), dtype=torch.float16, device="cuda") for _ in range(2)]
        return wsw.PagedKV(*kv, *(sc if cache == "q8_0" else (None, None)))
    rope = wsw.rope_table(d)
    x = torch.randn(n * length, 3 * h, d, generator=g).cuda()
    q, k, v = x.split([h, h, h], 1)
    pos = torch.arange(length).repeat(n)
    r = torch.arange(n).repeat_interleave(length)
    res = []
    for count, ids in ((6, torch.arange(6)), (pages, torch.tensor([0, pages - 1, pages // 2, pages - 2, 1, pages - 3]))):
        kv = make(count)
        table = ids.view(3, 2).to(torch.int32)
        slots = table[r, pos // page].long() * page + pos % page
        turned = wsw.rope_kv_write(q, k, v, rope, pos.to(torch.int32).cuda(), slots.cuda(), kv)
        lens = torch.full((n,), length, dtype=torch.int32, device="cuda")
        res.append((turned, wsw.attn_paged_decode(turned[length - 1::length].contiguous(), kv, table.cuda(), lens)))
        del kv
    assert res[1][1].isfinite().all()
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
