"""The streaming form of the rotary write (many aligned rows of 1024 tokens and more): q in place, launch
options, slots past the cache and padding, against the plain bounds and against itself bit for bit."""
import pytest
import torch

from helpers import need_gpu
from test_gpu_rope_kv import DT, _check, _make_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x,cache", [("bf16", "bf16"), ("fp16", "q8_0"), ("fp32", "q8_0")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_slots_past_the_cache_and_padding(x, cache, interleaved):
    wsw = need_gpu()
    tokens, page = 1500, 16
    room = (-(-tokens // page) + 2) * page
    g = torch.Generator().manual_seed(3)
    slots = torch.randperm(room, generator=g)[:tokens]
    positions = torch.randint(0, 70000, (tokens,), generator=g)
    slots[::7] = -1
    positions[3::50] = -4
    _check(wsw, x, cache, tokens, 20, 4, 128, 128, interleaved, page=page, slots=slots.clone(), positions=positions)
    slots[5::90] = room
    slots[6::300] = 1 << 40
    for opts in (None, {"pdl": 1}):
        _check(wsw, x, cache, tokens, 20, 4, 128, 128, interleaved, page=page, slots=slots.clone(), positions=positions,
               opts=opts)


@pytest.mark.parametrize("x,cache", [("bf16", "fp16"), ("fp16", "fp16"), ("fp32", "q8_0")])
@pytest.mark.parametrize("rot", [128, 64])
def test_q_in_place_and_launch_options(x, cache, rot):
    wsw = need_gpu()
    g = torch.Generator().manual_seed(5)
    tokens = 1111
    q = torch.randn(tokens, 24, 128, generator=g).to(DT[x]).cuda()
    k = torch.randn(tokens, 2, 128, generator=g).to(DT[x]).cuda()
    pos = torch.randint(0, 9999, (tokens,), generator=g).to(torch.int32).cuda()
    slots = torch.arange(tokens, device="cuda")
    kvs = [_make_cache(wsw, cache, 70, 16, 2, 128, True) for _ in range(3)]
    table = wsw.rope_table(rot)
    want = wsw.rope_kv_write(q, k, k, table, pos, slots, kvs[0])
    again = wsw.rope_kv_write(q, k, k, table, pos, slots, kvs[1], opts={"pdl": 1})
    own = q.clone()
    assert wsw.rope_kv_write(own, k, k, table, pos, slots, kvs[2], out=own, opts={"pdl": 1}) is own
    assert torch.equal(want, again) and torch.equal(want, own)
    for kv in kvs[1:]:
        for name in ("k", "v", "kd", "vd"):
            a, b = getattr(kvs[0], name), getattr(kv, name)
            assert a is None or torch.equal(a, b)
