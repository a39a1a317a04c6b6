"""Attention over shared prefixes in batches whose first rows are unused or shorter than the prefix."""
import pytest
import torch

from helpers import need_gpu
from test_gpu_attn_prefix import Case, _lens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("short", [[0], [0] * 31, [0] * 32 + [99], [0, 5, 99] * 700, [0] * 3000])
def test_a_group_whose_first_rows_are_short(short):
    c = Case(need_gpu(), [(100, short + _lens(100, 3, 60) + [0, 50]), (64, [0] * 40 + _lens(64, 0, 9)), (80, short)], kvh=1, group=2,
             d=64, behind=[5])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(err_flag=err)
    assert int(err) == 0


def test_many_groups_of_short_first_rows():
    c = Case(need_gpu(), [(20 + g % 40, [g % 19] * (g % 5) + _lens(20 + g % 40, 1, g % 3)) for g in range(700)], kvh=1, group=1, d=64,
             q="fp16", cache="fp16")
    c.check()


def test_heads_and_groups_near_the_limit():
    """11900 KV heads and room for 16384 groups, of which one has requests: within the stated limit for 32 positions."""
    c = Case(need_gpu(), [(8, [10, 12])], kvh=11900, group=1, d=64, q="fp16", cache="fp16")
    assert c.table.shape[1] * c.page == 32
    c.cu_d = torch.cat([c.cu_d, c.cu_d[-1:].expand(16383)]).contiguous()
    c.prefix_d = torch.cat([c.prefix_d, c.prefix_d.expand(16383)]).contiguous()
    c.check()
