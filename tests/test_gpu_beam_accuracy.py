"""What a beam's log softmax is off by, against 64 bits.

A row's sum is off by its terms' powers (2^-22 of each) and exponents (2 2^-24 |t| ln 2), of which a row behind a peak has
next to nothing, and by a tile's additions: of the peak's tile 15 at most, half a last place of 1 each (2^-24): 15 2^-24 in
all, and all downward where the other values are smaller than that.  Those are 15 exp(x - peak) in the mean, 15 e^(1/2 - peak) for
values of a normal distribution: 5.1e-8 for a peak of 20, and behind a row's other roundings, which have either sign, below
1e-7 in the mean over some hundred rows.  Any row: 2^-22 + 15 2^-24 + 26 2 2^-24 ln 2 < 2^-18."""
import numpy as np
import pytest
import torch

from helpers import need_gpu
from test_gpu_beam_select import T, _logits

pytestmark = pytest.mark.gpu


def _lse_errors(wsw, x, scale=1.0):
    """The best candidate's score less what it is in 64 bits, for each row: one beam a request."""
    r = wsw.beam_select(x, torch.zeros(len(x), 1, device="cuda"), scale=scale)
    y = x.double() * scale
    want = (y.max(-1).values - torch.logsumexp(y, -1)).cpu().numpy()
    got = r.score[:, 0].double().cpu().numpy()
    return got - want, 2.0 ** -24 * np.abs(want)


@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("place", ["first", "last", "middle", "any"])
@pytest.mark.parametrize("rows", [3, 320])
def test_rows_behind_a_peak(kind, place, rows):
    wsw = need_gpu()
    vocab = 152064
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, vocab, generator=g, device="cuda")
    at = {"first": 0, "last": vocab - 1, "middle": vocab // 2,
          "any": torch.randint(0, vocab, (rows,), generator=g, device="cuda")}[place]
    x[torch.arange(rows, device="cuda"), at] = 20 + torch.arange(rows, device="cuda").float() % 2
    err, rounding = _lse_errors(wsw, x.to(T[kind]))
    assert (np.abs(err) <= 15 * 2.0 ** -24 + 2.0 ** -26 + rounding).all(), np.abs(err).max()
    if rows > 100:
        assert abs(err.mean()) <= 1e-7, err.mean()


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("scale", [0.3, 1.0, 1.25, 7.0])
@pytest.mark.parametrize("rows,vocab", [(5, 50021), (400, 50021)])
def test_any_rows(kind, scale, rows, vocab):
    wsw = need_gpu()
    x = _logits(rows, rows, 1, vocab, kind).view(rows, vocab)
    x[1::5] = x[1::5].float().sort(-1).values.to(x.dtype)  # slowly rising rows: the maximum moves all the way
    x[2::5] = (x[2::5].float() * 0.01).to(x.dtype)
    x[3::5, 100:] -= 30
    x[4::5, ::7] = -float("inf")
    err, rounding = _lse_errors(wsw, x, scale)
    assert (np.abs(err) <= 2.0 ** -18 + rounding).all(), np.abs(err).max()
