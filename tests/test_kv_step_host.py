"""Host side of the paged-cache operators: argument checks (refused before any CUDA call),
workspace sizes, and the rotary frequency table against its formulas."""
import ctypes
import math

import numpy as np
import pytest

import kv_step_ref as ref
import weight_streaming_warp_gb300 as wsw

INVALID, MISALIGNED, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4
P = ctypes.c_void_p
A = P(4096)


@pytest.fixture(scope="module")
def lib():
    from weight_streaming_warp_gb300 import build
    build.build()
    return wsw.load()


def _cache(**kw):
    c = wsw._CKv(4096, 4096, None, None, 16, 16, 4, 128, 8192, 512, 128, 0, 0, 0, 1)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [
    (dict(k=None), INVALID), (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(heads=0), INVALID),
    (dict(pos_stride=-8), INVALID), (dict(page_size=24), UNSUPPORTED), (dict(page_size=1 << 17), UNSUPPORTED),
    (dict(head_dim=96), UNSUPPORTED), (dict(dtype=0), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED),
    (dict(num_pages=1 << 31), UNSUPPORTED), (dict(k=4104), MISALIGNED), (dict(head_stride=132), MISALIGNED),
    (dict(dtype=3), INVALID),  # q8_0 without scales
    (dict(dtype=3, kd=4096, vd=4100, d_page_stride=64, d_pos_stride=16, d_head_stride=4), MISALIGNED),
    (dict(dtype=3, kd=4096, vd=4096, d_page_stride=64, d_pos_stride=16, d_head_stride=2), MISALIGNED),
]


def _rope(lib, cache=None, q=A, k=A, dtype=0, tokens=2, heads=8, ts=1024, rot=128, inter=0, mscale=1.0, pos=A, slots=A,
          out=A, turns=A):
    return lib.wsw_rope_kv_write(q, k, A, dtype, tokens, heads, ts, 128, ts, 128, ts, 128, turns, rot, mscale, inter, pos,
                                 slots, out, ctypes.byref(cache or _cache()), None, None, None)


def _attn(lib, cache=None, q=A, dtype=0, n=2, heads=32, table=A, pages=8, ts=8, lens=A, scale=0.1, cap=0.0, window=0,
          out=A, ws=A, wsn=1 << 30):
    return lib.wsw_attn_paged_decode(q, dtype, n, heads, ctypes.byref(cache or _cache()), table, pages, ts, lens, scale,
                                     cap, window, None, out, None, None, ws, wsn, None, None)


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_bad_caches_are_refused(lib, change, status):
    assert _rope(lib, _cache(**change)) == status
    assert _attn(lib, _cache(**change)) == status


def test_rope_refusals(lib):
    assert _rope(lib, dtype=3) == UNSUPPORTED
    assert _rope(lib, rot=130) == INVALID and _rope(lib, rot=63) == INVALID
    assert _rope(lib, inter=2) == INVALID
    assert _rope(lib, mscale=math.inf) == INVALID
    assert _rope(lib, tokens=-1) == INVALID
    assert _rope(lib, tokens=1 << 31) == UNSUPPORTED
    assert _rope(lib, k=None) == INVALID and _rope(lib, q=None) == INVALID and _rope(lib, pos=None) == INVALID
    assert _rope(lib, turns=None) == INVALID
    assert _rope(lib, q=P(4098)) == MISALIGNED and _rope(lib, slots=P(4100)) == MISALIGNED
    assert _rope(lib, tokens=0, q=None, k=None) == 0


def test_attention_refusals(lib):
    assert _attn(lib, dtype=3) == UNSUPPORTED
    assert _attn(lib, heads=30) == INVALID  # not a multiple of 4 KV heads
    assert _attn(lib, heads=0) == INVALID and _attn(lib, n=-1) == INVALID
    assert _attn(lib, scale=math.nan) == INVALID and _attn(lib, cap=-1.0) == INVALID and _attn(lib, window=-1) == INVALID
    assert _attn(lib, ts=4) == INVALID  # a row shorter than max_pages
    assert _attn(lib, n=70000) == UNSUPPORTED and _attn(lib, window=1 << 31) == UNSUPPORTED
    assert _attn(lib, pages=1 << 28, ts=1 << 28) == UNSUPPORTED  # 2^32 positions
    big = _cache(page_size=65536, heads=64)
    assert _attn(lib, cache=big, heads=64, n=60000, pages=1024, ts=1024) == UNSUPPORTED  # 2^34 tiles
    assert _attn(lib, q=None) == INVALID and _attn(lib, ws=None) == INVALID and _attn(lib, table=None) == INVALID
    assert _attn(lib, q=P(4104)) == MISALIGNED and _attn(lib, lens=P(4097)) == MISALIGNED
    assert _attn(lib, wsn=1000) == WORKSPACE
    assert _attn(lib, n=0, q=None) == 0
    wb = lib.wsw_attn_paged_decode_workspace_bytes
    # counters, and 132 floats per query row for two records of each of 152 CTAs and one of each warp
    assert wb(1, 32, 4, 128) == 2048 + 152 * 14 * 8 * 132 * 4
    assert wb(64, 40, 4, 128) == 2048 + 152 * 14 * 16 * 132 * 4
    assert wb(64, 40, 4, 256) == 2048 + 152 * 6 * 16 * 260 * 4
    assert wb(1, 30, 4, 128) == 0 and wb(1, 32, 4, 96) == 0


def test_plan_refusals(lib):
    def plan(seq=A, n=4, nfree=8, page=16, pages=8, ts=8, tokens=4, pos=A, slots=A, head=A, free=A):
        return lib.wsw_kv_page_plan(seq, A, n, free, nfree, head, page, A, pages, ts, tokens, pos, slots, A, A, A, None,
                                    None, None)
    assert plan(n=-1) == INVALID and plan(nfree=-1) == INVALID and plan(tokens=-1) == INVALID
    assert plan(page=0) == INVALID and plan(page=12) == UNSUPPORTED and plan(page=1 << 17) == UNSUPPORTED
    assert plan(ts=4) == INVALID
    assert plan(n=20000) == UNSUPPORTED
    assert plan(seq=None) == INVALID and plan(head=None) == INVALID and plan(free=None) == INVALID
    assert plan(slots=P(4100)) == MISALIGNED and plan(seq=P(4097)) == MISALIGNED


def test_logprobs_refusals(lib):
    def lp(x=A, dtype=0, rows=2, vocab=100, ld=100, tokens=A, scale=1.0, top=5, out=A, rank=A, ws=None, wsn=0, ids=A):
        return lib.wsw_token_logprobs(x, dtype, rows, vocab, ld, tokens, scale, top, out, rank, A, A, A, ids, ws, wsn,
                                      None, None)
    assert lp(dtype=3) == UNSUPPORTED and lp(top=33) == UNSUPPORTED
    assert lp(vocab=4, top=5) == INVALID and lp(ld=99) == INVALID and lp(vocab=0) == INVALID and lp(top=-1) == INVALID
    assert lp(scale=0.0) == INVALID and lp(scale=-1.0) == INVALID and lp(scale=math.inf) == INVALID
    assert lp(tokens=None) == INVALID and lp(rank=None) == INVALID and lp(ids=None) == INVALID and lp(x=None) == INVALID
    assert lp(x=P(4098)) == MISALIGNED and lp(x=P(4097), dtype=2) == MISALIGNED
    assert lp(rows=1, vocab=152064, ld=152064) == WORKSPACE
    assert lp(rows=1, vocab=152064, ld=152064, ws=P(4104), wsn=1 << 20) == MISALIGNED
    assert lp(rows=0, x=None) == 0
    wb = lib.wsw_token_logprobs_workspace_bytes
    assert wb(5000, 152064, 20) == 0 and wb(1, 100, 20) == 0 and wb(1, 152064, 20) > 0 and wb(0, 10, 0) == 0


@pytest.mark.parametrize("rot,theta,scaling,factor,original", [
    (128, 10000.0, None, 1.0, 0), (64, 500000.0, "linear", 8.0, 0), (96, 10000.0, "ntk", 4.0, 0),
    (128, 10000.0, "by_parts", 4.0, 32768), (2, 100.0, None, 1.0, 0), (256, 1e6, "by_parts", 40.0, 4096)])
def test_rope_table_follows_its_formulas(lib, rot, theta, scaling, factor, original):
    t = wsw.rope_table(rot, theta, scaling, factor, original, device="cpu")
    f, m = ref.rope_freqs(rot, theta, scaling, factor, original)
    turns = t.turns.numpy().view(np.uint64)
    # whole numbers of 2^-64 turns, from doubles with a handful of roundings of 2^-53 on each side
    want = f / (2 * math.pi) * 2.0 ** 64
    assert np.all(np.abs(turns.astype(np.float64) - want) <= 0.5 + 1e-14 * want)
    assert abs(t.mscale - m) <= 2.0 ** -24 * m and t.rot_dim == rot
    assert np.all(np.diff(f) < 0) or rot == 2


def test_rope_table_takes_frequencies_and_refuses(lib):
    f = [1.0, 0.25, 1e-6, 0.0]
    t = wsw.rope_table(8, freqs=f, device="cpu")
    want = np.array(f) / (2 * math.pi) * 2.0 ** 64
    assert np.all(np.abs(t.turns.numpy().view(np.uint64).astype(np.float64) - want) <= 0.5 + 1e-15 * want)
    assert t.mscale == 1.0
    for bad in (dict(rot_dim=7), dict(rot_dim=258), dict(rot_dim=8, theta=1.0), dict(rot_dim=2, scaling="ntk", factor=2.0),
                dict(rot_dim=8, scaling="linear", factor=0.5), dict(rot_dim=8, scaling="by_parts", factor=2.0),
                dict(rot_dim=4, freqs=[1.0, 7.0]), dict(rot_dim=4, freqs=[1.0, math.nan]), dict(rot_dim=4, freqs=[1.0]),
                dict(rot_dim=8, scaling="other")):
        with pytest.raises(wsw.WswError):
            wsw.rope_table(device="cpu", **bad)


def test_binding_refuses_host_tensors():
    import torch
    x = torch.zeros(2, 4, 128)
    for call in (lambda: wsw.PagedKV(x, x), lambda: wsw.token_logprobs(torch.zeros(2, 8)),
                 lambda: wsw.kv_page_plan(torch.zeros(2, dtype=torch.int32), None, None, None, None, 16, 4)):
        with pytest.raises(wsw.WswError):
            call()


# 2 pi to 60 digits
TWO_PI = "6.28318530717958647692528676655900576839433879875021164194989"


@pytest.mark.parametrize("rot,theta,scaling,factor,original", [
    (128, 10000.0, None, 1.0, 0), (256, 1e6, None, 1.0, 0), (2, 100.0, None, 1.0, 0), (64, 500000.0, "linear", 8.0, 0),
    (96, 1234.5, "linear", 3.7, 0), (128, 10000.0, "ntk", 4.0, 0), (4, 10000.0, "ntk", 2.5, 0), (250, 1e6, "ntk", 16.0, 0),
    (128, 10000.0, "by_parts", 4.0, 32768), (256, 1e6, "by_parts", 40.0, 4096), (64, 1.0000001, None, 1.0, 0),
    (128, 1e300, None, 1.0, 0),
    (6, 1e308, "ntk", 1e100, 0)])
def test_rope_table_against_40_digits(lib, rot, theta, scaling, factor, original):
    """The table is the definition's turns rounded to whole 2^-64 turns, so that position times
    turns is off by half a position 2^-64 turns: 7e-10 radians at position 2^31.  (Frequencies in
    doubles are off by f 2^-53 or more: 3e-7 radians there.)"""
    import decimal
    with decimal.localcontext(decimal.Context(prec=50)):
        D = decimal.Decimal
        two_pi, unit = D(TWO_PI), D(2) ** 64
        t = wsw.rope_table(rot, theta, scaling, factor, original, device="cpu")
        got = [int(x) for x in t.turns.numpy().view(np.uint64)]
        for i in range(rot // 2):
            base = D(theta) * (D(factor) ** (D(rot) / D(rot - 2)) if scaling == "ntk" else 1)
            f = base ** (D(-2 * i) / D(rot))
            if scaling == "linear":
                f /= D(factor)
            if scaling == "by_parts":
                keep = min(max((D(original) * f / two_pi - 1) / 31, D(0)), D(1))
                f = keep * f + (1 - keep) * f / D(factor)
            # beside the rounding, 2^-90 of the value for the way there
            assert abs(got[i] - f / two_pi * unit) <= D(0.5) + D(2) ** -90 * unit, i


def test_own_frequencies_against_40_digits(lib):
    import decimal
    f = [6.28, 1.0, 0.3, 1e-3, 1e-9, 2.0 ** -60, 5e-324, 0.0]
    t = wsw.rope_table(16, freqs=f, device="cpu")
    with decimal.localcontext(decimal.Context(prec=50)):
        D = decimal.Decimal
        for got, want in zip(t.turns.numpy().view(np.uint64), f):
            assert abs(int(got) - D(want) / D(TWO_PI) * D(2) ** 64) <= D(0.5) + D(2) ** -26


def test_attention_refuses_tables_that_reach_two_to_the_31(lib):
    """Tiles and windows of the table run past the last position: 2^31 - 4096 of them at most."""
    most = (1 << 31) - 4096
    for page, pages in ((1, most + 1), (1, (1 << 31) - 1), (8, (1 << 28) - 1), (16, (1 << 27) - 255), (4096, 1 << 19)):
        assert pages * page > most
        assert _attn(lib, cache=_cache(page_size=page), pages=pages, ts=pages, window=1) == UNSUPPORTED
    for page, pages in ((1, most), (16, (1 << 27) - 256), (4096, (1 << 19) - 1)):  # the next refusal, as they pass this one
        assert pages * page <= most
        assert _attn(lib, cache=_cache(page_size=page), pages=pages, ts=pages, window=1, q=None) == INVALID


def test_plan_refuses_tokens_that_reach_two_to_the_31(lib):
    """Threads step in rounds of up to 65536 places past the last token: 2^31 - 2^20 at most."""
    def plan(tokens, seq=A):
        return lib.wsw_kv_page_plan(seq, A, 4, A, 8, A, 16, A, 8, 8, tokens, A, A, A, A, A, None, None, None)
    most = (1 << 31) - (1 << 20)
    for tokens in (most + 1, (1 << 31) - 3, (1 << 31) - 2):
        assert plan(tokens) == UNSUPPORTED
    assert plan(most, seq=P(4097)) == MISALIGNED  # the next refusal


def test_scales_whose_log2_form_overflows_are_refused(lib):
    """scale * log2 e has to be finite, too: 0 times an infinite one is NaN."""
    for scale in (3.4e38, -3.4e38, 2.4e38):
        assert _attn(lib, scale=scale) == INVALID
    assert _attn(lib, scale=2.3e38, lens=P(4097)) == MISALIGNED and _attn(lib, scale=-2.3e38, lens=P(4097)) == MISALIGNED

    def lp(scale, x=A):
        return lib.wsw_token_logprobs(x, 0, 2, 100, 100, A, scale, 5, A, A, A, A, A, A, None, 0, None, None)
    assert lp(3.4e38) == INVALID and lp(2.4e38) == INVALID and lp(2.3e38, x=P(4098)) == MISALIGNED


def test_attention_refuses_rows_beyond_32_bits(lib):
    """The zeros of a request of no tokens are counted in vectors of four with 32 bits."""
    one = _cache(heads=1, head_dim=256, pos_stride=256, head_stride=256)
    most = ((1 << 31) - 4096) // 64
    assert _attn(lib, cache=one, n=1, heads=most + 1) == UNSUPPORTED
    assert _attn(lib, cache=one, n=1, heads=most, q=None) == INVALID  # the next refusal
