"""Rows of logits with a NaN or +inf: every fp32 result of the row is NaN, its ids stay in range and
its neighbours do not change a bit.  The value sits in the row's unaligned beginning, inside a whole vector,
in its last values, or next to a split's edge, in each type, with one split and with several."""
import math

import pytest
import torch

from helpers import need_gpu

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.mark.parametrize("x", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("rows,vocab", [(3, 37), (3, 3001), (3, 20011), (400, 9003)])
def test_a_value_spoils_its_row_alone(x, value, rows, vocab):
    wsw = need_gpu()
    g = torch.Generator().manual_seed(vocab)
    ld = vocab + 3
    buf = torch.zeros(1 + rows * ld, dtype=DT[x], device="cuda")
    logits = buf[1:].view(rows, ld)[:, :vocab]  # no row begins on 16 bytes, or few
    clean = (torch.randn(rows, vocab, generator=g) * 3).to(DT[x]).cuda()
    tokens = torch.randint(0, vocab, (rows,), generator=g).to(torch.int32).cuda()
    for top in (5, 0, 20):
        logits.copy_(clean)
        want = wsw.token_logprobs(logits, tokens, top=top)
        for at in (0, 2, vocab // 2, 4096 % vocab, vocab - 2, vocab - 1):
            logits.copy_(clean)
            logits[1, at] = value
            got = wsw.token_logprobs(logits, tokens, top=top)
            for name, a, b in zip(got._fields, got, want):
                keep = torch.ones(rows, dtype=torch.bool, device="cuda")
                keep[1] = False
                assert torch.equal(a[keep], b[keep]), (name, at)
                if a.dtype == torch.float32:
                    assert torch.isnan(a[1]).all(), (name, at, a[1])
                elif a.numel():
                    assert int(a[1].min()) >= -1 and int(a[1].max()) < vocab, (name, at)
