"""Sines and cosines of rotary angles on the GPU against 64 bits.

A pair (1, 0) turns into (cos a, sin a) with no rounding of its own.  The angle is an exact
fraction of a turn, of which nothing is lost that fp32 could show; sincospif is off by one ulp at most
(2^-24 below 1) and the correction's sum rounds once more (2^-25)."""
import numpy as np
import pytest
import torch

from helpers import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form,tokens,heads", [("plain", 64, 2), ("plain", 3000, 2), ("streaming", 3000, 20)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("far", [4096, 1 << 31])
def test_sines_and_cosines_carry_fp32(form, tokens, heads, interleaved, far):
    wsw = need_gpu()
    g = torch.Generator().manual_seed(tokens + heads)
    pos = torch.randint(0, far, (tokens,), generator=g)
    pos[:5] = torch.tensor([0, 1, 2, 3, far - 1])
    x = torch.zeros(tokens, heads + 4, 128, device="cuda")
    x[..., slice(0, 128, 2) if interleaved else slice(0, 64)] = 1.0
    q, k, v = x.split([heads, 2, 2], 1)
    pages = -(-tokens // 16)
    if form == "streaming":  # fp32 rows take it into q8_0 pages, from 1024 tokens of 24 rows on
        kv = wsw.PagedKV(*[torch.zeros(pages, 16, 2, 128, dtype=torch.int8, device="cuda") for _ in range(2)],
                         *[torch.zeros(pages, 16, 2, 4, dtype=torch.float16, device="cuda") for _ in range(2)])
    else:
        kv = wsw.PagedKV(*[torch.zeros(pages, 16, 2, 128, dtype=torch.float16, device="cuda") for _ in range(2)])
    table = wsw.rope_table(128)
    out = wsw.rope_kv_write(q, k, v, table, pos.to(torch.int32).cuda(), torch.arange(tokens).cuda(), kv,
                            interleaved=interleaved).double().cpu().numpy()
    turns = table.turns.cpu().numpy().view(np.uint64)
    part = (pos.numpy().astype(np.uint64)[:, None] * turns).view(np.int64).astype(np.longdouble) / 2 ** 63  # half turns
    a = (part * np.pi).astype(np.float64)[:, None]
    cos, sin = (out[..., 0::2], out[..., 1::2]) if interleaved else (out[..., :64], out[..., 64:])
    lim = 1.5 * 2.0 ** -24 + 2.0 ** -40
    assert np.abs(cos - np.cos(a)).max() <= lim
    assert np.abs(sin - np.sin(a)).max() <= lim
