"""Page plan on the GPU against the plain loop: whole numbers, equal everywhere."""
import numpy as np
import pytest
import torch

import kv_step_ref as ref
from helpers import need_gpu

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _case(seed, n, cached, new, page, width=None, zero=0.2):
    g = np.random.default_rng(seed)
    seq = g.integers(0, cached + 1, n)
    add = g.integers(0, 2 * new + 1, n) * (g.random(n) > zero)
    width = width or -(-(cached + 2 * new) // page)
    have = -(-seq // page)
    total = int(have.sum())
    need = int((-(-(seq + add) // page) - have).sum())
    ids = g.permutation(total + need + 5)
    table = np.full((n, width), -1)
    at = 0
    for r in range(n):
        table[r, :have[r]] = ids[at: at + have[r]][:width]
        at += have[r]
    return seq, add, ids[total:], table


def _check(wsw, seq, add, free, table, page, tokens, head=0, in_place=False, opts=None):
    want = ref.page_plan(seq, add, free, head, table, page, tokens)
    seq_d, add_d, free_d, head_d, table_d = _i32(seq), _i32(add), _i32(free), _i32([head]), _i32(table)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = None
    if in_place:
        out = (torch.full((tokens,), 77, dtype=torch.int32, device="cuda"),
               torch.full((tokens,), 77, dtype=torch.int64, device="cuda"),
               torch.full((len(seq) + 1,), 77, dtype=torch.int32, device="cuda"), seq_d, head_d)
    p = wsw.kv_page_plan(seq_d, add_d, free_d, head_d, table_d, page, tokens, out=out, err_flag=err, opts=opts)
    for name, got, exp in (("table", table_d, want[0]), ("positions", p.positions, want[1]), ("slots", p.slots, want[2]),
                           ("cu", p.cu, want[3]), ("seq_len", p.seq_len, want[4]), ("head", p.head, [want[5]]),
                           ("err", err, [want[6]])):
        assert np.array_equal(got.cpu().numpy(), np.asarray(exp)), name
    return want


@pytest.mark.parametrize("n,cached,new,page", [
    (1, 0, 1, 16), (1, 5, 1, 1), (3, 100, 0, 16), (64, 4096, 1, 16), (65, 1000, 40, 8), (129, 50, 3, 256),
    (1000, 4096, 70, 32), (1025, 100, 20, 16), (4097, 64, 2, 64), (16384, 9, 1, 4), (7, 20000, 9000, 65536)])
@pytest.mark.parametrize("in_place", [False, True])
def test_matches_the_plain_loop(n, cached, new, page, in_place):
    wsw = need_gpu()
    seq, add, free, table = _case(n + page, n, cached, new, page)
    tokens = int(add.sum()) + (n % 3) * 5  # some padding rows
    want = _check(wsw, seq, add, free, table, page, tokens, in_place=in_place)
    assert want[6] == 0


@pytest.mark.parametrize("what", ["pages", "width", "tokens", "negative", "bad head", "all"])
@pytest.mark.parametrize("n", [5, 300])
def test_requests_that_do_not_fit(what, n):
    wsw = need_gpu()
    seq, add, free, table = _case(n, n, 200, 30, 8)
    tokens, head = int(add.sum()) + 2, 0
    if what in ("pages", "all"):
        free = free[: max(1, len(free) // 2)]
    if what in ("width", "all"):
        table = table[:, : table.shape[1] // 2]
    if what in ("tokens", "all"):
        tokens = tokens // 2
    if what in ("negative", "all"):
        seq[1], add[2] = -3, -1
    if what == "bad head":
        head = len(free) + 1
    want = _check(wsw, seq, add, free, table, 8, tokens, head=head)
    assert want[6] != 0


def test_empty_and_offset_free_list():
    wsw = need_gpu()
    _check(wsw, np.zeros(0, int), np.zeros(0, int), np.arange(4), np.zeros((0, 4), int), 16, 3)
    seq, add, free, table = _case(9, 40, 100, 10, 16)
    _check(wsw, seq, add, np.concatenate([np.full(7, 99), free]), table, 16, int(add.sum()), head=7, opts={"pdl": 1})


def test_negative_table_entries_give_no_slot():
    wsw = need_gpu()
    seq, add, free, table = _case(11, 20, 100, 10, 16)
    table[:10] = -1
    _check(wsw, seq, add, free, table, 16, int(add.sum()))


def test_strided_table_and_graph_replay():
    """A captured plan advances lengths, list and table in place at each replay."""
    wsw = need_gpu()
    n, page, steps = 33, 4, 9
    big = torch.full((n, 20), -1, dtype=torch.int32, device="cuda")
    table = big[:, :10]
    lens, one = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.ones(n, dtype=torch.int32, device="cuda")
    g = np.random.default_rng(3)
    ids = g.permutation(n * 10)
    free, head = _i32(ids), _i32([0])
    out = (torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.int64, device="cuda"),
           torch.empty(n + 1, dtype=torch.int32, device="cuda"), lens, head)
    wsw.kv_page_plan(lens, one, free, head, table, page, n, out=out)  # warm-up: the first step
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wsw.kv_page_plan(lens, one, free, head, table, page, n, out=out)
    hl, hh, ht = np.zeros(n, int), 0, np.full((n, 10), -1)
    for step in range(steps):
        ht, pos, slot, cu, hl, hh, err = ref.page_plan(hl, np.ones(n, int), ids, hh, ht, page, n)
        if step:
            graph.replay()
        assert np.array_equal(out[0].cpu().numpy(), pos) and np.array_equal(out[1].cpu().numpy(), slot), step
        assert np.array_equal(lens.cpu().numpy(), hl) and int(head) == hh
    assert np.array_equal(table.cpu().numpy(), ht) and int(big[:, 10:].max()) == -1


def test_slots_past_32_bits():
    wsw = need_gpu()
    seq, add = np.array([70000, 0, 65535]), np.array([3, 2, 2])
    table = np.full((3, 3), -1)
    table[0, :2], table[2, 0] = [1 << 30, (1 << 31) - 1], (1 << 31) - 2
    want = _check(wsw, seq, add, np.array([1 << 29, (1 << 31) - 3]), table, 65536, 8)
    assert want[6] == 0 and want[2].max() > 1 << 46
