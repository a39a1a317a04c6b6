"""What the binding's calls for rows that share pages refuse before the library is called, without a
GPU: host tensors that say they are on a device stand in for device tensors."""
import pytest
import torch

import weight_streaming_warp_gb300 as wsw
from test_kv_binding_host import I32, I64, U8, calls, stand  # noqa: F401  (a fixture)

F32 = torch.float32


def i(*shape, **kw):
    return stand(*shape, dtype=kw.pop("dtype", I32), **kw)


def copies(n=4, fill=True, **kw):
    return wsw.PageCopies(i(n, **kw), i(n, **kw), i(n, **kw) if fill else None, i(1, **kw))


def cache(index=0):
    return wsw.PagedKV(*[stand(3, 16, 2, 64, dtype=torch.float16, index=index) for _ in range(2)])


def refused(call, calls, *words):  # noqa: F811
    del calls[:]
    with pytest.raises(wsw.WswError) as e:
        call()
    assert calls == [] and all(w in str(e.value) for w in words), e.value


def test_handles_check_their_tensors(calls):  # noqa: F811
    table = i(4, 8)
    for make in (lambda: wsw.PageCopies(torch.zeros(4, dtype=I32), i(4), i(4), i(1)),
                 lambda: wsw.PageCopies(i(4), i(5), i(4), i(1)),
                 lambda: wsw.PageCopies(i(4), i(4), i(3), i(1)),
                 lambda: wsw.PageCopies(i(4), i(4), i(4), i(2)),
                 lambda: wsw.PageCopies(i(4, dtype=I64), i(4), i(4), i(1)),
                 lambda: wsw.PageCopies(i(8)[::2], i(4), i(4), i(1)),
                 lambda: wsw.PageCopies(i(4), i(4, index=1), i(4), i(1)),
                 lambda: wsw.KvFork(table, i(5), i(1), copies(5)),
                 lambda: wsw.KvFork(table, i(4), i(2), copies()),
                 lambda: wsw.KvFork(table, i(4), i(1), copies(3)),
                 lambda: wsw.KvFork(table, i(4), i(1), copies(fill=False)),
                 lambda: wsw.KvFork(table, i(4), i(1), copies(index=1)),
                 lambda: wsw.KvFork(i(4, 8, index=1), i(4), i(1), copies()),
                 lambda: wsw.KvCompact(table, i(9), i(2), copies(0, False)),
                 lambda: wsw.KvCompact(table, i(9), i(1), copies(0, True)),
                 lambda: wsw.KvCompact(i(32), i(9), i(1), copies(0, False)),
                 lambda: wsw.BeamStep(i(2, 3), i(2, 3), i(2, 3), i(2, 3), i(2, 3), stand(2, 3)),
                 lambda: wsw.BeamStep(i(2, 3), i(2, 3), stand(2, 3), i(2, 3), i(2, 4), stand(2, 3))):
        refused(make, calls)
    c = copies()
    with pytest.raises(AttributeError):
        c.src = i(4)
    assert [x is y for x, y in zip(c, (c.src, c.dst, c.fill, c.count))] == [True] * 4


def _fork(out=None, **change):
    a = dict(parent=i(4), seq_len=i(3), free_pages=i(9), head=i(1), table=i(3, 8), page_size=16, err_flag=i(1))
    a.update(change)
    return wsw.kv_page_fork(out=out or wsw.KvFork(i(4, 8), i(4), i(1), copies()), **a)


def test_fork(calls):  # noqa: F811
    _fork()
    assert calls == ["wsw_kv_page_fork"]
    for change in (dict(parent=torch.zeros(4, dtype=I32)), dict(parent=i(4, dtype=I64)), dict(seq_len=i(4)),
                   dict(free_pages=i(9, index=1)), dict(head=i(2)), dict(table=i(3, 9)), dict(table=i(3, 8, index=1)),
                   dict(parent=i(5)), dict(err_flag=i(1, dtype=I64)),
                   dict(out=wsw.KvFork(i(4, 8, index=1), i(4, index=1), i(1, index=1), copies(index=1)))):
        refused(lambda: _fork(**change), calls)


def test_copy(calls):  # noqa: F811
    wsw.kv_page_copy(copies(), cache())
    wsw.kv_page_copy(copies(fill=False), [cache(), cache()], err_flag=i(1))
    assert calls == ["wsw_kv_page_copy"] * 2
    refused(lambda: wsw.kv_page_copy(copies(), [cache(), cache(1)]), calls)
    refused(lambda: wsw.kv_page_copy(copies(index=1), cache(1)), calls)  # the current device is another one
    refused(lambda: wsw.kv_page_copy(copies(), cache(), err_flag=i(1, index=1)), calls)


def _compact(n=3, pages=9, moves=2, **change):
    a = dict(seq_len=i(3), table=i(3, 8), page_size=16, num_pages=9, held=i(9, dtype=U8), max_moves=2,
             ws=i(64, dtype=U8), err_flag=i(1))
    a.update(change)
    out = wsw.KvCompact(i(n, 8), i(pages), i(1), copies(moves, False))
    return wsw.kv_page_compact(out=out, **a)


def test_compact(calls):  # noqa: F811
    _compact()
    assert calls == ["wsw_kv_page_compact"]
    for change in (dict(n=4), dict(pages=8), dict(moves=3), dict(held=i(8, dtype=U8)), dict(held=i(9)), dict(ws=i(64)),
                   dict(ws=i(64, dtype=U8, index=1)), dict(seq_len=i(4)), dict(table=i(3, 7))):
        refused(lambda: _compact(**change), calls)


def _beam(**change):
    a = dict(logits=stand(6, 50), scores=stand(2, 3), end_tokens=[1], ws=i(64, dtype=U8),
             out=wsw.BeamStep(i(2, 3), i(2, 3), stand(2, 3), i(2, 3), i(2, 3), stand(2, 3)))
    a.update(change)
    return wsw.beam_select(**a)


def test_beam_select(calls):  # noqa: F811
    _beam()
    assert calls == ["wsw_beam_select"]
    wide = wsw.BeamStep(i(3, 2), i(3, 2), stand(3, 2), i(3, 2), i(3, 2), stand(3, 2))
    for change in (dict(logits=torch.zeros(6, 50)), dict(logits=stand(6, 50, dtype=torch.float64)), dict(logits=stand(7, 50)),
                   dict(logits=stand(50, 6).T), dict(scores=stand(6)), dict(scores=stand(2, 3, index=1)),
                   dict(scores=stand(2, 3, dtype=torch.float16)), dict(out=wide), dict(ws=i(64))):
        refused(lambda: _beam(**change), calls)


def _attend(**change):
    a = dict(q=stand(4, 8, 64), kv=cache(), table=i(4, 2), lens=i(4), groups=i(3), prefix=i(2), out=stand(4, 8, 64),
             lse=stand(4, 8), slopes=stand(8), ws=i(64, dtype=U8), err_flag=i(1))
    a.update(change)
    return wsw.attn_paged_prefix(**a)


def test_prefix_attention(calls):  # noqa: F811
    _attend()
    assert calls == ["wsw_attn_paged_prefix"]
    for change in (dict(q=stand(4, 8, 128)), dict(q=stand(4, 7, 64)), dict(q=stand(4, 64)), dict(kv=cache(1)),
                   dict(q=stand(8, 4, 64).transpose(0, 1)), dict(table=i(5, 2)), dict(lens=i(5)), dict(groups=i(2)),
                   dict(groups=i(3, dtype=I64)), dict(prefix=i(3)), dict(out=stand(4, 8, 64, dtype=torch.float16)),
                   dict(lse=stand(4, 7)), dict(slopes=stand(7)), dict(ws=i(64)), dict(ws=i(64, dtype=U8, index=1))):
        refused(lambda: _attend(**change), calls)
