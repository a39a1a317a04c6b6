"""Rotary positions and the paged cache write on the GPU against the formulas in 64 bits.

Tolerance of a rotated value m (x0 cos a - x1 sin a): the angle in half turns is rounded to
fp32 (2^-24 of at most one half turn: pi 2^-24 radians) after a cut at 2^-32 turns; sine and
cosine (2 ulp: 2^-22 at most), the factor, two products and a sum (2^-24 each) follow.  In
all less than (pi + 4 + 3 + 0.1) 2^-24 < 11 2^-24 times m (|x0| + |x1|), plus half a step of
the stored type.  q8_0: the code of a value that far from the exact one can differ by one
step where x / d is near a half, so a stored value is within half a step d of the exact
value, plus the same error and the scale's rounding to binary16 (2^-11 of the value)."""
import numpy as np
import pytest
import torch

import kv_step_ref as ref
from helpers import need_gpu

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
STEP = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"fp32": 0.0, "fp16": 2.0 ** -25, "bf16": 0.0}  # half a subnormal step


def _np(t):
    return t.double().cpu().numpy()


def _make_cache(wsw, cache, pages, page, h, d, nhd, fill=0.0):
    shape = (pages, page, h) if nhd else (pages, h, page)
    if cache == "q8_0":
        kv = [torch.full((*shape, d), 3, dtype=torch.int8, device="cuda") for _ in range(2)]
        sc = [torch.full((*shape, d // 32), 0.5, dtype=torch.float16, device="cuda") for _ in range(2)]
    else:
        kv = [torch.full((*shape, d), fill, dtype=DT[cache], device="cuda") for _ in range(2)]
        sc = [None, None]
    return wsw.PagedKV(kv[0], kv[1], sc[0], sc[1], layout="nhd" if nhd else "hnd")


def _rows(kv, i):
    """K (0) or V (1) as [slots][heads][dim] float64, and the scales [slots][heads][dim / 32]."""
    x, s = (kv.k, kv.kd) if i == 0 else (kv.v, kv.vd)
    if kv.layout == "hnd":
        x = x.transpose(1, 2)
        s = s.transpose(1, 2) if s is not None else None
    x = _np(x.reshape(-1, kv.heads, kv.head_dim))
    if s is None:
        return x, None
    s = _np(s.reshape(-1, kv.heads, kv.head_dim // 32))
    return x * np.repeat(s, 32, -1), s


def _check(wsw, x, cache, tokens, hq, h, d, rot, interleaved, page=16, nhd=True, scaling=None, far=4096, slots=None,
           positions=None, fused=True, offset=0, opts=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    width = (hq + 2 * h) * d
    raw = torch.randn(tokens, width + offset, generator=g).to(DT[x]).cuda()
    qkv = raw[:, offset:].unflatten(1, (hq + 2 * h, d))
    q, k, v = qkv.split([hq, h, h], 1)
    if not fused:
        q, k, v = q.contiguous(), k.transpose(0, 1).contiguous().transpose(0, 1), v.contiguous()
    pages = -(-tokens // page) + 2
    if slots is None:
        slots = torch.randperm(pages * page, generator=g)[:tokens]
    if positions is None:
        positions = torch.randint(0, far, (tokens,), generator=g)
    kw = dict(scaling=scaling, factor=4.0, original=1024) if scaling else {}
    table = wsw.rope_table(rot, **kw)
    kv = _make_cache(wsw, cache, pages, page, h, d, nhd)
    before = [_rows(kv, i)[0] for i in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = wsw.rope_kv_write(q, k, v, table, positions.to(torch.int32).cuda(), slots.cuda(), kv, interleaved=interleaved,
                            err_flag=err, opts=opts)
    pos, sl = positions.numpy(), slots.numpy()
    f, m = ref.rope_freqs(rot, **kw)
    live = pos >= 0

    def turned(t):
        a = _np(t)
        y = ref.rotate(a, np.maximum(pos, 0), f, m, interleaved)
        mag = np.abs(a).copy()
        r = 2 * len(f)
        if interleaved:
            s = mag[..., 0:r:2] + mag[..., 1:r:2]
            mag[..., :r] = np.repeat(s, 2, -1) * m
        else:
            s = mag[..., : r // 2] + mag[..., r // 2: r]
            mag[..., :r] = np.concatenate([s, s], -1) * m
        bound = 11 * 2.0 ** -24 * mag
        bound[..., r:] = 0  # copied
        y[~live] = 0
        bound[~live] = 0
        return y, bound

    yq, bq = turned(q)
    assert (np.abs(_np(out) - yq) <= bq + STEP[x] * (np.abs(yq) + bq) + TINY[x]).all(), "q"
    room = pages * page
    ok = live & (sl >= 0) & (sl < room)
    assert int(err) == int((live & (sl >= room)).any())
    for i, (src, name) in enumerate(((k, "k"), (v, "v"))):
        y, b = turned(src) if i == 0 else (_np(src), np.zeros(src.shape))
        got, sc = _rows(kv, i)
        untouched = np.ones(room, bool)
        untouched[sl[ok]] = False
        assert np.array_equal(got[untouched], before[i][untouched]), name + ": other rows"
        gy, y, b = got[sl[ok]], y[ok], b[ok]
        if cache == "q8_0":
            blocks = np.abs(y).reshape(*y.shape[:2], -1, 32).max(-1) / 127
            db = b.reshape(*y.shape[:2], -1, 32).max(-1) / 127
            ds = sc[sl[ok]]
            assert (np.abs(ds - blocks) <= db + (2.0 ** -11 + 2.0 ** -23) * blocks + 2.0 ** -25).all(), name + ": scales"
            step = np.repeat(blocks + db, 32, -1)
            lim = 0.5 * step * (1 + 2.0 ** -20) + b + 127 * np.repeat(db, 32, -1) + (np.abs(y) + step) * 2.0 ** -11 \
                + 127 * 2.0 ** -25
            assert (np.abs(gy - y) <= lim).all(), name
        else:
            assert (np.abs(gy - y) <= b + STEP[cache] * (np.abs(y) + b) + TINY[cache]).all(), name
    return out, kv


@pytest.mark.parametrize("x,cache", [("fp32", "fp16"), ("fp32", "bf16"), ("fp32", "q8_0"), ("bf16", "bf16"),
                                     ("bf16", "q8_0"), ("fp16", "fp16"), ("fp16", "q8_0"), ("bf16", "fp16")])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (256, 128), (128, 40), (64, 20), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_types_widths_and_pairings(x, cache, d, rot, interleaved):
    wsw = need_gpu()
    if rot == 0:
        rot = 2  # one pair only
    _check(wsw, x, cache, 37, 6, 2, d, rot, interleaved, nhd=interleaved)


@pytest.mark.parametrize("x,cache", [("bf16", "bf16"), ("fp16", "q8_0"), ("fp32", "q8_0"), ("fp32", "fp16")])
@pytest.mark.parametrize("hq,h,d,rot,interleaved", [
    (20, 4, 128, 128, False), (20, 2, 128, 96, True), (40, 4, 64, 64, False), (8, 2, 256, 256, False), (24, 1, 128, 40, False),
    (1, 1, 64, 64, False), (1, 1, 128, 40, True), (3, 1, 128, 128, False), (8, 2, 64, 32, False), (2, 1, 256, 64, True)])
@pytest.mark.parametrize("tokens", [1024, 2435])
def test_prompts_of_many_and_few_heads(x, cache, hq, h, d, rot, interleaved, tokens):
    wsw = need_gpu()
    g = torch.Generator().manual_seed(tokens)
    slots = torch.randperm(-(-tokens // 16) * 16 + 32, generator=g)[:tokens]
    positions = torch.randint(0, 100000, (tokens,), generator=g)
    unused = torch.rand(tokens, generator=g) < 0.05
    slots[unused], positions[unused] = -1, -1
    _check(wsw, x, cache, tokens, hq, h, d, rot, interleaved, nhd=tokens == 1024, slots=slots, positions=positions)


@pytest.mark.parametrize("tokens", [1, 2, 255, 2047, 2049, 4099])
def test_token_counts(tokens):
    wsw = need_gpu()
    _check(wsw, "fp32", "fp16", tokens, 5, 1, 128, 128, False, page=64, nhd=False)
    _check(wsw, "bf16", "q8_0", tokens, 3, 3, 64, 32, True, page=1)


@pytest.mark.parametrize("hq,h", [(40, 4), (32, 4), (0, 2), (1, 1), (128, 8)])
def test_head_counts(hq, h):
    wsw = need_gpu()
    _check(wsw, "fp32", "q8_0", 9, hq, h, 128, 128, False)


@pytest.mark.parametrize("scaling", ["linear", "ntk", "by_parts"])
def test_scalings_and_far_positions(scaling):
    wsw = need_gpu()
    far = torch.tensor([0, 1, 131071, 1 << 20, (1 << 24) + 1, (1 << 30) + 12345, (1 << 31) - 1])
    # the table's frequencies carry 2^-53 of relative rounding and 2^-65 turns of absolute: at
    # 2^31 positions below 2^-21 radians in all, as large as the fp32 steps; so near positions
    # are held to the formula and far ones to the table's own angles
    _check(wsw, "fp32", "fp16", 5, 4, 2, 128, 128, False, scaling=scaling, positions=far[:5])
    table = wsw.rope_table(64, scaling=scaling, factor=4.0, original=1024)
    t = table.turns.cpu().numpy().view(np.uint64)
    frac = (far.numpy().astype(np.uint64)[:, None] * t[None, :]).astype(np.float64) / 2.0 ** 64
    kv = _make_cache(wsw, "fp16", 3, 16, 1, 64, True)
    q = torch.zeros(7, 1, 64, device="cuda")
    q[..., :32] = 1.0
    out = wsw.rope_kv_write(q, q, q, table, far.to(torch.int32).cuda(), torch.arange(7).cuda(), kv)
    got = _np(out)[:, 0]
    assert (np.abs(got[:, :32] - table.mscale * np.cos(2 * np.pi * frac)) <= 11 * 2.0 ** -24 * table.mscale).all()
    assert (np.abs(got[:, 32:] - table.mscale * np.sin(2 * np.pi * frac)) <= 11 * 2.0 ** -24 * table.mscale).all()


@pytest.mark.parametrize("fused,offset", [(True, 0), (False, 0), (True, 1), (True, 4)])
@pytest.mark.parametrize("x", ["fp32", "bf16"])
def test_strides_and_alignment(fused, offset, x):
    wsw = need_gpu()
    a, kva = _check(wsw, x, "fp16", 33, 4, 2, 128, 64, False, fused=fused, offset=offset)
    _check(wsw, x, "q8_0", 33, 4, 2, 128, 128, True, fused=fused, offset=offset)


def test_padding_and_slots_outside_the_cache():
    wsw = need_gpu()
    tokens, page = 12, 16
    slots = torch.tensor([0, 5, -1, 17, 48, 1 << 40, -9, 30, 31, 2, 3, 4])  # 3 pages of 16
    pos = torch.tensor([3, 0, 7, -1, 9, 10, -5, 11, 100, 2, 1, 5])
    for cache in ("fp16", "q8_0"):
        _check(wsw, "fp32", cache, tokens, 4, 2, 128, 128, False, page=page, slots=slots, positions=pos)
    _check(wsw, "fp32", "fp16", tokens, 4, 2, 128, 128, False, page=page,
           slots=torch.where(slots >= 48, torch.tensor(-1), slots), positions=pos)


def test_q_in_place_and_launch_options():
    wsw = need_gpu()
    g = torch.Generator().manual_seed(5)
    q = torch.randn(300, 8, 128, generator=g).cuda()
    k = torch.randn(300, 2, 128, generator=g).cuda()
    pos, slots = torch.arange(300, dtype=torch.int32, device="cuda"), torch.arange(300, device="cuda")
    kv = _make_cache(wsw, "bf16", 20, 16, 2, 128, True)
    table = wsw.rope_table(128)
    a = wsw.rope_kv_write(q, k, k, table, pos, slots, kv)
    for opts in ({"pdl": 1}, {"ctas_per_sm": 1}):
        b = wsw.rope_kv_write(q, k, k, table, pos, slots, kv, opts=opts)
        assert torch.equal(a, b)
    q2 = q.clone()
    assert wsw.rope_kv_write(q2, k, k, table, pos, slots, kv, out=q2) is q2
    assert torch.equal(a, q2)


def test_q8_codes_equal_the_quantizer_where_nothing_rotates():
    """V is not rotated: its codes and scales are those of quantize_q8, bit for bit."""
    wsw = need_gpu()
    g = torch.Generator().manual_seed(6)
    v = (torch.randn(50, 4, 128, generator=g) * torch.exp(3 * torch.randn(50, 4, 1, generator=g))).cuda()
    v[7] = 0
    kv = _make_cache(wsw, "q8_0", 4, 16, 4, 128, True)
    pos, slots = torch.arange(50, dtype=torch.int32, device="cuda"), torch.arange(50, device="cuda")
    wsw.rope_kv_write(v, v, v, wsw.rope_table(128), pos, slots, kv)
    codes, scales = wsw.quantize_q8(v.view(200, 128), 32)
    assert torch.equal(kv.v.view(-1, 128)[:200], codes)
    assert torch.equal(kv.vd.view(-1, 4)[:200].view(torch.int16), scales.view(torch.int16))
