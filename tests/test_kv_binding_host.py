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
    monkeypatch.setattr(wsw, "_stream", lambda: 0)
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
