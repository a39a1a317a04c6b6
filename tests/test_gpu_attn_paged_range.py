"""Paged decode attention at the ends of its types' ranges, against the formula in 64 bits (the
inputs, bounds and check of test_gpu_attn_paged)."""
import pytest
import torch

from helpers import need_gpu
from test_gpu_attn_paged import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,group,q", [(128, 4, "bf16"), (64, 10, "fp32"), (256, 1, "bf16"), (128, 16, "bf16")])
def test_bf16_values_near_the_largest(d, group, q):
    """Values up to 2^125: a weighted sum of them overflows only where weights grow past 1."""
    wsw = need_gpu()
    c = Case(wsw, [1, 2, 40, 300], group=group, d=d, q=q, cache="bf16")
    c.kv.v.copy_(c.kv.v.double() * 2.0 ** 122)
    c.vals[1] *= 2.0 ** 122
    c.check()
