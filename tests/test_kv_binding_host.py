"""What the paged-cache calls of the binding refuse before the library is called, without a
GPU: host tensors that say they are on a device stand in for device tensors, and a recorder
for the library."""
import types

import pytest
import torch

import weight_streaming_warp_gb300 as wsw

I32, I64, U8 = torch.int32, torch.int64, torch.uint8


class Stand(torch.Tensor):
    """A host tensor that claims to be on cuda:`index`."""
    index = 0

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cuda", self.index)

    def get_device(self):
        return self.index


def stand(*shape, dtype=torch.float32, index=0):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(Stand)
    t.index = index
    return t


@pytest.fixture
def calls(monkeypatch):
    """The names of the library calls made."""
    made = []

    class Library:
        def __getattr__(self, name):
            if name.endswith("_workspace_bytes"):
                return lambda *a: 64
            return lambda *a: made.append(name) or 0

    monkeypatch.setattr(wsw, "load", Library)
    monkeypatch.setattr(wsw, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(wsw, "_current_device", lambda: 0)
    return made


def _rope(rope=None, **change):
    t = dict(q=stand(5, 8, 64), k=stand(5, 2, 64), v=stand(5, 2, 64), positions=stand(5, dtype=I32),
             slots=stand(5, dtype=I64), kv=wsw.PagedKV(stand(3, 16, 2, 64, dtype=torch.float16),
                                                       stand(3, 16, 2, 64, dtype=torch.float16)),
             out=stand(5, 8, 64), err_flag=stand(1, dtype=I32))
    t.update(change)
    args = types.SimpleNamespace(**t)
    rope = wsw.RopeTable(stand(32, dtype=I64), 1.0, 64) if rope is None else rope
    return wsw.rope_kv_write(args.q, args.k, args.v, rope, args.positions, args.slots, args.kv, out=args.out,
                             err_flag=args.err_flag)


def test_rope_takes_a_device_table_of_its_size_only(calls):
    _rope()
    _rope(wsw.RopeTable(stand(0, dtype=I64), 1.0, 0))
    assert calls == ["wsw_rope_kv_write"] * 2
    del calls[:]
    for turns, rot in ((torch.zeros(32, dtype=I64), 64),      # a host table
                       (stand(31, dtype=I64), 64),            # shorter than rot_dim / 2
                       (stand(32, dtype=I64), 128),
                       (stand(32, dtype=torch.float64), 64),
                       (stand(64, dtype=I64)[::2], 64),       # not contiguous
                       (None, 64)):
        with pytest.raises(wsw.WswError, match="rope.turns"):
            _rope(wsw.RopeTable(turns, 1.0, rot))
    assert calls == []


def _plan(change):
    t = dict(seq_len=stand(4, dtype=I32), new_len=stand(4, dtype=I32), free_pages=stand(9, dtype=I32),
             head=stand(1, dtype=I32), table=stand(4, 3, dtype=I32), positions=stand(6, dtype=I32),
             slots=stand(6, dtype=I64), cu=stand(5, dtype=I32), lens=stand(4, dtype=I32), head_out=stand(1, dtype=I32),
             err_flag=stand(1, dtype=I32))
    t.update(change)
    return wsw.kv_page_plan(t["seq_len"], t["new_len"], t["free_pages"], t["head"], t["table"], 16, 6,
                            out=tuple(t[n] for n in ("positions", "slots", "cu", "lens", "head_out")),
                            err_flag=t["err_flag"])


def _cache(change, dtype=torch.int8):
    t = dict(k=stand(3, 16, 2, 64, dtype=dtype), v=stand(3, 16, 2, 64, dtype=dtype))
    if dtype == torch.int8:
        t.update(kd=stand(3, 16, 2, 2, dtype=torch.float16), vd=stand(3, 16, 2, 2, dtype=torch.float16))
    t.update(change)
    return wsw.PagedKV(**t)


def _attn(change):
    t = dict(q=stand(4, 6, 64), table=stand(4, 3, dtype=I32), lens=stand(4, dtype=I32), slopes=stand(6),
             out=stand(4, 6, 64), lse=stand(4, 6), err_flag=stand(1, dtype=I32), ws=stand(64, dtype=U8))
    t.update(change)
    kv = t.pop("kv", None) or _cache({})
    return wsw.attn_paged_decode(t.pop("q"), kv, t.pop("table"), t.pop("lens"), **t)


def _logprobs(change):
    t = dict(logits=stand(4, 50), tokens=stand(4, dtype=I32), ws=stand(64, dtype=U8), logprob=stand(4),
             rank=stand(4, dtype=I32), lse=stand(4), entropy=stand(4), top_logprob=stand(4, 2),
             top_id=stand(4, 2, dtype=I32))
    t.update(change)
    out = tuple(t[n] for n in ("logprob", "rank", "lse", "entropy", "top_logprob", "top_id"))
    return wsw.token_logprobs(t["logits"], t["tokens"], top=2, out=out, ws=t["ws"])


def _write(change):
    change = dict(change)
    turns = change.pop("turns", None)
    return _rope(None if turns is None else wsw.RopeTable(turns, 1.0, 64), **change)


ELSEWHERE = [
    (_plan, "wsw_kv_page_plan", dict(
        seq_len=(4, I32), new_len=(4, I32), free_pages=(9, I32), head=(1, I32), table=(4, 3, I32), positions=(6, I32),
        slots=(6, I64), cu=(5, I32), lens=(4, I32), head_out=(1, I32), err_flag=(1, I32))),
    (_write, "wsw_rope_kv_write", dict(
        q=(5, 8, 64), k=(5, 2, 64), v=(5, 2, 64), positions=(5, I32), slots=(5, I64), out=(5, 8, 64), err_flag=(1, I32),
        turns=(32, I64))),
    (_attn, "wsw_attn_paged_decode", dict(
        q=(4, 6, 64), table=(4, 3, I32), lens=(4, I32), slopes=(6,), out=(4, 6, 64), lse=(4, 6), err_flag=(1, I32),
        ws=(64, U8))),
    (_logprobs, "wsw_token_logprobs", dict(
        logits=(4, 50), tokens=(4, I32), ws=(64, U8), logprob=(4,), rank=(4, I32), lse=(4,), entropy=(4,),
        top_logprob=(4, 2), top_id=(4, 2, I32))),
]


def _on(index, spec):
    spec = list(spec)
    dtype = spec.pop() if isinstance(spec[-1], torch.dtype) else torch.float32
    return stand(*spec, dtype=dtype, index=index)


@pytest.mark.parametrize("call,name,tensors", ELSEWHERE, ids=[n for _, n, _ in ELSEWHERE])
def test_tensors_of_another_device_are_refused(calls, monkeypatch, call, name, tensors):
    """A launch is the current device's: an address of another one would be followed there."""
    call({})
    assert calls == [name]
    del calls[:]
    for which, spec in tensors.items():
        with pytest.raises(wsw.WswError, match="device"):
            call({which: _on(1, spec)})
    monkeypatch.setattr(wsw, "_current_device", lambda: 1)
    with pytest.raises(wsw.WswError, match="device"):
        call({})
    if "out" in tensors:  # a cache, of one device or of two
        monkeypatch.setattr(wsw, "_current_device", lambda: 0)
        other = [stand(3, 16, 2, 64, dtype=torch.int8, index=1) for _ in range(2)]
        scales = [stand(3, 16, 2, 2, dtype=torch.float16, index=1) for _ in range(2)]
        with pytest.raises(wsw.WswError, match="device"):
            call({"kv": wsw.PagedKV(*other, *scales)})
        for i, part in enumerate(("k", "v", "kd", "vd")):
            with pytest.raises(wsw.WswError, match="device"):
                _cache({part: (other + scales)[i]})
    assert calls == []
