"""What the calls for rows that share pages refuse on the host, before anything is launched."""
import ctypes

import pytest

import weight_streaming_warp_gb300 as wsw

INVALID, MISALIGNED, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4
P, N = ctypes.c_void_p, None
A = P(4096)


@pytest.fixture(scope="module")
def lib():
    from weight_streaming_warp_gb300 import build
    build.build()
    return wsw.load()


def _fork(lib, **change):
    a = dict(parent=P(1 << 20), children=4, seq=P(2 << 20), requests=4, free=A, n_free=8, head=A, page=16,
             table=P(3 << 20), width=8, stride=8, out=P(4 << 20), out_stride=8, lens=P(5 << 20), head_out=A, src=A, dst=A,
             fill=A, count=A, err=N)
    a.update(change)
    return lib.wsw_kv_page_fork(*a.values(), None, None)


def test_fork_rejects_on_host(lib):
    for name in ("parent", "seq", "free", "head", "table", "out", "lens", "head_out", "src", "dst", "fill", "count"):
        assert _fork(lib, **{name: N}) == INVALID, name
        assert _fork(lib, **{name: P((6 << 20) + 2)}) == MISALIGNED, name
    assert _fork(lib, err=P(4098)) == MISALIGNED
    for change in ({"children": -1}, {"requests": -1}, {"n_free": -1}, {"width": -1}, {"page": 0}, {"stride": 7},
                   {"out_stride": 7}):
        assert _fork(lib, **change) == INVALID, change
    for change in ({"children": 8193}, {"requests": 8193}, {"page": 48}, {"page": 1 << 17}, {"n_free": (1 << 31) - 1},
                   {"width": 1 << 31, "stride": 1 << 31, "out_stride": 1 << 31}, {"stride": 1 << 50},
                   {"out_stride": 1 << 50}):
        assert _fork(lib, **change) == UNSUPPORTED, change
    # the new table overlaps the old one, but is not the old one; the lengths likewise
    assert _fork(lib, out=P((3 << 20) + 4)) == INVALID
    assert _fork(lib, out=P(3 << 20), out_stride=9) == INVALID
    assert _fork(lib, out=P((3 << 20) - 4 * 8 * 4 + 4)) == INVALID
    assert _fork(lib, lens=P((2 << 20) + 4)) == INVALID


def _cache(**change):
    c = dict(k=4096, v=4096, kd=None, vd=None, num_pages=8, page_size=16, heads=2, head_dim=64, page_stride=2048,
             pos_stride=128, head_stride=64, d_page_stride=0, d_pos_stride=0, d_head_stride=0, dtype=1)
    c.update(change)
    return wsw._CKv(**c)


def _copy(lib, *caches, src=A, dst=A, fill=A, count=A, copies=4, n=None, err=N):
    refs = (P * max(1, len(caches)))(*[ctypes.addressof(c) if c else None for c in caches])
    return lib.wsw_kv_page_copy(src, dst, fill, count, copies, refs, len(caches) if n is None else n, err, None, None)


def test_copy_rejects_on_host(lib):
    ok = _cache()
    assert _copy(lib) == 0 and _copy(lib, ok, copies=0, src=N, dst=N, count=N) == 0
    for name in ("src", "dst", "count"):
        assert _copy(lib, ok, **{name: N}) == INVALID
        assert _copy(lib, ok, **{name: P(4098)}) == MISALIGNED
    assert _copy(lib, ok, fill=P(4097)) == MISALIGNED and _copy(lib, ok, err=P(4097)) == MISALIGNED
    assert _copy(lib, ok, copies=-1) == INVALID and _copy(lib, ok, n=-1) == INVALID
    assert _copy(lib, ok, copies=1 << 31) == UNSUPPORTED
    assert _copy(lib, ok, _cache(page_size=8)) == INVALID  # one block table, one page size
    assert _copy(lib, ok, None) == INVALID
    assert _copy(lib, ok, _cache(k=4104)) == MISALIGNED
    assert _copy(lib, ok, _cache(head_dim=96)) == UNSUPPORTED
    assert _copy(lib, ok, _cache(dtype=3)) == INVALID  # q8_0 without scales
    assert lib.wsw_kv_page_copy(A, A, N, A, 4, None, 1, N, None, None) == INVALID


def _compact(lib, **change):
    a = dict(seq=A, requests=4, table=P(3 << 20), width=8, stride=8, page=16, pool=100, held=N, moves=5, out=P(4 << 20),
             out_stride=8, free=A, head=A, src=A, dst=A, count=A, err=N, ws=A, ws_bytes=1 << 20)
    a.update(change)
    return lib.wsw_kv_page_compact(*a.values(), None, None)


def test_compact_rejects_on_host(lib):
    for name in ("seq", "table", "out", "free", "head", "src", "dst", "count", "ws"):
        assert _compact(lib, **{name: N}) == INVALID, name
    for name in ("seq", "table", "out", "free", "head", "src", "dst", "count", "err", "ws"):
        assert _compact(lib, **{name: P((6 << 20) + 2)}) == MISALIGNED, name
    for change in ({"requests": -1}, {"width": -1}, {"stride": 7}, {"out_stride": 7}, {"page": 0}, {"pool": 0},
                   {"moves": -1}, {"out": P((3 << 20) + 4)}, {"out": P(3 << 20), "out_stride": 9}):
        assert _compact(lib, **change) == INVALID, change
    for change in ({"requests": 65536}, {"page": 24}, {"page": 1 << 17}, {"pool": (1 << 22) + 1}, {"moves": 1 << 31},
                   {"stride": 1 << 50}, {"width": 1 << 31, "stride": 1 << 31, "out_stride": 1 << 31}):
        assert _compact(lib, **change) == UNSUPPORTED, change
    need = lib.wsw_kv_page_compact_workspace_bytes
    assert need(0) == 0 and need((1 << 22) + 1) == 0 and need(100) >= 100 + 400
    assert _compact(lib, ws_bytes=need(100) - 1) == WORKSPACE


def _beam(lib, **change):
    a = dict(logits=A, dtype=0, requests=2, beams=4, vocab=1000, ld=1000, scores=A, ends=(ctypes.c_int32 * 1)(5), n_ends=1,
             scale=ctypes.c_float(1.0), parent=A, token=A, score=A, end_parent=A, end_token=A, end_score=A, ws=A,
             ws_bytes=1 << 24)
    a.update(change)
    return lib.wsw_beam_select(*a.values(), None, None)


def test_beam_select_rejects_on_host(lib):
    for name in ("logits", "scores", "ends", "parent", "token", "score", "end_parent", "end_token", "end_score", "ws"):
        assert _beam(lib, **{name: N}) == INVALID, name
    assert _beam(lib, end_parent=N, end_token=N, end_score=N) == INVALID  # there is an end token
    for name in ("logits", "scores", "parent", "token", "score", "end_parent", "end_token", "end_score", "ws"):
        assert _beam(lib, **{name: P((1 << 20) + 2)}) == MISALIGNED, name
    assert _beam(lib, logits=P(4097), dtype=1) == MISALIGNED
    for change in ({"requests": -1}, {"beams": 0}, {"vocab": 0}, {"ld": 999}, {"n_ends": -1}, {"scale": ctypes.c_float(0)},
                   {"scale": ctypes.c_float(-1)}, {"scale": ctypes.c_float(float("nan"))},
                   {"scale": ctypes.c_float(3e38)}):
        assert _beam(lib, **change) == INVALID, change
    for change in ({"dtype": 3}, {"requests": 16385}, {"beams": 33, "n_ends": 0}, {"beams": 17}, {"n_ends": 9, "beams": 1},
                   {"vocab": (1 << 31) - 65536, "ld": 1 << 31}):
        assert _beam(lib, **change) == UNSUPPORTED, change
    need = lib.wsw_beam_select_workspace_bytes
    assert need(0, 4, 10, 0) == 0 and need(1, 33, 10, 0) == 0 and need(1, 16, 1000, 2) == 0
    assert _beam(lib, ws_bytes=need(2, 4, 1000, 1) - 1) == WORKSPACE
    assert _beam(lib, requests=0, logits=N, ws=N) == 0


def _attend(lib, **change):
    c = _cache()
    a = dict(q=A, dtype=2, requests=4, q_heads=8, cache=ctypes.byref(c), table=A, width=8, stride=8, lens=A, cu=A, groups=2,
             prefix=A, share=1, scale=ctypes.c_float(0.1), softcap=ctypes.c_float(0), slopes=N, out=A, lse=N, err=N, ws=A,
             ws_bytes=1 << 40)
    a.update(change)
    return lib.wsw_attn_paged_prefix(*a.values(), None, None)


def test_attn_prefix_rejects_on_host(lib):
    for name in ("q", "cache", "table", "lens", "cu", "prefix", "out", "ws"):
        assert _attend(lib, **{name: N}) == INVALID, name
    for name in ("q", "table", "lens", "cu", "prefix", "slopes", "out", "lse", "err", "ws"):
        assert _attend(lib, **{name: P(4098)}) == MISALIGNED, name
    for change in ({"requests": -1}, {"q_heads": 7}, {"groups": 0}, {"groups": -1}, {"share": 2}, {"stride": 7}, {"width": -1},
                   {"scale": ctypes.c_float(float("inf"))}, {"softcap": ctypes.c_float(-1)}):
        assert _attend(lib, **change) == INVALID, change
    for change in ({"dtype": 3}, {"requests": 65536}, {"groups": 16385}, {"cache": ctypes.byref(_cache(head_dim=256))},
                   {"requests": 60000, "q_heads": 32768}, {"width": 1 << 27, "stride": 1 << 27},
                   {"groups": 16384, "width": 1 << 20, "stride": 1 << 20}):
        assert _attend(lib, **change) == UNSUPPORTED, change
    assert _attend(lib, ws=P(4096 + 128)) == MISALIGNED
    need = lib.wsw_attn_paged_prefix_workspace_bytes
    assert need(4, 0, 8, 2, 64) == 0 and need(4, 2, 8, 2, 256) == 0 and need(4, 16385, 8, 2, 64) == 0
    assert _attend(lib, ws_bytes=need(4, 2, 8, 2, 64) - 1) == WORKSPACE
    assert _attend(lib, requests=0, q=N, out=N, ws=N) == 0
