"""Token log probabilities on the GPU against the definition in 64 bits.

Tolerances, with n = vocab and eps = 2^-24.  An exponential 2^d has a relative error of
2^-22 (ex2) plus |d| times the rounding of d (2 eps, ln 2); weighted by 2^d this stays below
2^-21 of the largest term.  A thread adds at most n / 256 + 4 terms, each sum off by eps, and
about 16 joins follow: sums are within S_REL = 2^-21 + (n / 256 + 20) eps.  So ln S, and with
the roundings of (x - m) scale and the last sum: |lse|, |logprob| errors within S_REL + 3 eps
(|value| + |ln S| + |x_t - m| scale).  The entropy ln S - E / S: E's terms have one sign and
the same errors, so within S_REL (1 + 2 |E / S|) + 3 eps (|ln S| + |E / S|)."""
import math

import numpy as np
import pytest
import torch

import kv_step_ref as ref
from helpers import need_gpu

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 2.0 ** -24


def _check(wsw, logits, tokens, top, scale, ws=None, opts=None):
    """logits: a device tensor [rows][vocab] of any row stride."""
    rows, vocab = logits.shape
    r = wsw.token_logprobs(logits, None if tokens is None else torch.tensor(tokens, dtype=torch.int32, device="cuda"),
                           top=top, scale=scale, ws=ws, opts=opts)
    x = logits.double().cpu().numpy()
    got = {k: getattr(r, k).double().cpu().numpy() for k in ("lse", "entropy", "top_logprob")}
    ids = r.top_id.cpu().numpy()
    s_rel = 2.0 ** -21 + (vocab / 256 + 20) * EPS
    for i in range(rows):
        t = 0 if tokens is None else tokens[i]
        inside = 0 <= t < vocab
        lp, rank, lse, ent, order, best, ln_s = ref.logprobs(x[i], t if inside else 0, scale, top)
        assert np.array_equal(ids[i], order), i
        if tokens is not None:
            assert int(r.rank[i]) == (rank if inside else -1)
        if lse == -math.inf:
            assert got["lse"][i] == -math.inf and got["entropy"][i] == 0 and (got["top_logprob"][i] == -math.inf).all()
            if tokens is not None:
                assert float(r.logprob[i]) == -math.inf
            continue
        m = x[i].max() * scale
        assert abs(got["lse"][i] - lse) <= s_rel + 3 * EPS * (abs(lse) + abs(ln_s) + abs(m)), i
        mean = abs(ln_s - ent)
        assert abs(got["entropy"][i] - ent) <= s_rel * (1 + 2 * mean) + 3 * EPS * (abs(ln_s) + mean), i
        for value, exact in ([(got["top_logprob"][i], best)] +
                             ([(np.array([float(r.logprob[i])]), np.array([lp]))] if tokens is not None and inside
                              else [])):
            fin = np.isfinite(exact)
            assert np.array_equal(np.isfinite(value), fin) and (value[~fin] == -math.inf).all()
            lim = s_rel + 3 * EPS * (np.abs(exact[fin]) + abs(ln_s) + np.abs(exact[fin] + ln_s))
            assert (np.abs(value[fin] - exact[fin]) <= lim).all(), i
        if tokens is not None and not inside:
            assert math.isnan(float(r.logprob[i]))
    return r


def _normal(seed, rows, vocab, dtype, sigma=2.5):
    return (torch.randn(rows, vocab, generator=torch.Generator().manual_seed(seed)) * sigma).to(DT[dtype]).cuda()


@pytest.mark.parametrize("x", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (1, 7, 7), (3, 33, 32), (2, 1000, 20), (5, 8191, 5),
                                            (1, 152064, 20), (2, 50021, 32), (400, 4099, 1), (3, 65537, 0)])
def test_sizes_and_types(x, rows, vocab, top):
    wsw = need_gpu()
    g = np.random.default_rng(rows + vocab)
    _check(wsw, _normal(vocab, rows, vocab, x), [int(t) for t in g.integers(0, vocab, rows)], top, 1.0)


@pytest.mark.parametrize("x", ["fp32", "bf16"])
@pytest.mark.parametrize("scale", [0.01, 1.25, 40.0])
def test_scales_and_the_best_token(x, scale):
    wsw = need_gpu()
    lg = _normal(3, 4, 9001, x)
    best = lg.float().argmax(1).tolist()
    r = _check(wsw, lg, best, 8, scale)
    assert (r.rank == 0).all() and torch.equal(r.top_id[:, 0].cpu(), torch.tensor(best, dtype=torch.int32))
    assert torch.equal(r.logprob, r.top_logprob[:, 0])


@pytest.mark.parametrize("x", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("top", [1, 5, 20])
@pytest.mark.parametrize("rows", [1, 700])
def test_the_rows_last_values_tie_with_earlier_ones(x, top, rows):
    """The row's end, which no whole 16-byte vector holds, ranks after every equal value."""
    wsw = need_gpu()
    vocab = 33001
    lg = -1.0 - torch.rand(rows, vocab, generator=torch.Generator().manual_seed(8))
    lg[:, 100: 100 + top - 1] = 5.0
    lg[:, 2000:2400] = 2.0  # enough candidates for a cut before the tie is read
    lg[:, 30000] = 3.0
    lg[:, vocab - 1] = 3.0
    _check(wsw, lg.to(DT[x]).cuda(), [vocab - 1] * rows, top, 1.0)


@pytest.mark.parametrize("x", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("top", [1, 8, 32])
@pytest.mark.parametrize("rows", [2, 320])
@pytest.mark.parametrize("kind", ["islands", "drift", "steps"])
def test_uneven_rows_overflow_the_candidates(x, top, rows, kind):
    """Parts of a row far above what came before: more candidates at once than are kept."""
    wsw = need_gpu()
    vocab = 40009
    lg = torch.randn(rows, vocab, generator=torch.Generator().manual_seed(10)) * 2.5
    if kind == "islands":
        lg[:, 9000:11000] += 5.0
        lg[:, 26001:26002] = 40.0
        lg[:, 33333:40009] += 9.0
    elif kind == "drift":
        lg += torch.linspace(0, 20, vocab)
    else:
        lg = torch.arange(vocab).div(1500, rounding_mode="floor").float().expand(rows, vocab).clone()
    _check(wsw, lg.to(DT[x]).cuda(), [(1237 * i) % vocab for i in range(rows)], top, 1.0)


@pytest.mark.parametrize("offset,ld", [(0, 3001), (1, 3001), (3, 3007), (5, 4096)])
@pytest.mark.parametrize("x", ["fp32", "fp16"])
def test_strides_and_alignment(offset, ld, x):
    wsw = need_gpu()
    buf = torch.full((6 * ld + 64,), float("nan"), dtype=DT[x], device="cuda")
    view = buf[offset: offset + 6 * ld].view(6, ld)[:, :2999]
    view.copy_(_normal(4, 6, 2999, x))
    _check(wsw, view, [0, 1, 2998, 5, 1500, 7], 10, 1.0)
    one = buf[offset: offset + 2999].view(1, 2999)
    _check(wsw, one, [2998], 10, 1.0)


@pytest.mark.parametrize("vocab", [1000, 20000, 152064])
@pytest.mark.parametrize("rows", [1, 200])
def test_forbidden_tokens_and_rows_of_nothing_else(vocab, rows):
    wsw = need_gpu()
    if rows * vocab > 5_000_000:
        rows = 3
    lg = _normal(5, rows, vocab, "fp32")
    keep = torch.rand(rows, vocab, generator=torch.Generator().manual_seed(1)).cuda() < 0.3
    lg = lg.masked_fill(~keep, -math.inf)
    lg[0] = -math.inf
    if rows > 1:
        lg[1] = -math.inf
        lg[1, vocab - 2] = 1.5  # a single token left
    if rows > 2:
        lg[2] = torch.finfo(torch.float32).min  # all at the type's lowest value: uniform
    g = np.random.default_rng(6)
    _check(wsw, lg, [int(t) for t in g.integers(0, vocab, rows)], 20, 1.0)


@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "two values", "few levels", "lowest and one"])
@pytest.mark.parametrize("vocab", [500, 9000, 70000])
def test_ties_and_orders_that_fill_the_candidate_buffer(kind, vocab):
    wsw = need_gpu()
    i = torch.arange(vocab, dtype=torch.float32)
    x = {"equal": torch.zeros(vocab), "rising": i * 1e-3, "falling": -i * 1e-3,
         "two values": (i % 2), "few levels": torch.floor(torch.rand(vocab, generator=torch.Generator().manual_seed(2)) * 5),
         "lowest and one": torch.where(i == vocab // 2, 0.0, torch.finfo(torch.float32).min)}[kind]
    rows = x.repeat(2, 1).cuda()
    rows[1] *= 2
    for top in (1, 20, 32):
        _check(wsw, rows, [vocab - 1, vocab // 3], top, 1.0)
    many = x.repeat(310, 1).cuda()  # one CTA per row
    r = wsw.token_logprobs(many, top=32)
    order = torch.tensor(np.lexsort((np.arange(vocab), -x.numpy()))[:32].copy(), dtype=torch.int32)
    assert (r.top_id.cpu() == order).all()


def test_negative_zero_is_zero():
    wsw = need_gpu()
    x = torch.tensor([[-0.0, 0.0, -0.0, 0.0, -1.0]], device="cuda")
    r = _check(wsw, x, [3], 4, 1.0)
    assert r.top_id[0].tolist() == [0, 1, 2, 3] and int(r.rank) == 3


def test_nan_and_infinity_stay_in_their_rows():
    wsw = need_gpu()
    for vocab in (300, 40000):
        lg = _normal(7, 4, vocab, "fp32")
        lg[1, 5] = math.nan
        lg[2, vocab - 1] = math.inf
        t = torch.tensor([1, 2, 3, 4], dtype=torch.int32, device="cuda")
        r = wsw.token_logprobs(lg, t, top=5)
        for row in (1, 2):
            assert all(math.isnan(float(v[row])) for v in (r.lse, r.entropy, r.logprob)) or row == 2
            assert not math.isfinite(float(r.lse[row])) and math.isnan(float(r.entropy[row]))
        assert int(r.top_id.min()) >= -1 and int(r.top_id.max()) < vocab
        good = torch.tensor([0, 3], device="cuda")
        clean = wsw.token_logprobs(lg[good].contiguous(), t[good], top=5)
        for name in ("lse", "entropy", "logprob", "rank", "top_id"):
            a, b = getattr(r, name)[good], getattr(clean, name)
            assert torch.allclose(a.float(), b.float(), rtol=0, atol=1e-4), name


def test_tokens_outside_the_vocabulary():
    wsw = need_gpu()
    _check(wsw, _normal(8, 4, 1234, "bf16"), [-1, 1234, 1 << 30, 7], 3, 1.0)


def test_workspace_reuse_options_and_streams():
    wsw = need_gpu()
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    lg = _normal(9, 2, 152064, "fp32")
    a = _check(wsw, lg, [5, 6], 20, 1.0, ws=ws)
    for rows, vocab in ((1, 60000), (7, 30000), (2, 152064)):
        _check(wsw, _normal(10, rows, vocab, "bf16"), list(range(rows)), 7, 1.0, ws=ws)
    for opts in (None, {"pdl": 1}):
        b = _check(wsw, lg, [5, 6], 20, 1.0, ws=ws, opts=opts)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c = wsw.token_logprobs(lg, torch.tensor([5, 6], dtype=torch.int32, device="cuda"), top=20)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(a, c))
    torch.cuda.synchronize()
    assert int(ws[:2048].view(torch.int32).abs().sum()) == 0, "counters left nonzero"


def test_rows_past_32_bits():
    wsw = need_gpu()
    ld = (1 << 31) + 4096  # elements between rows
    buf = torch.empty(2 * ld, dtype=torch.bfloat16, device="cuda")
    view = buf.view(2, ld)[:, :20001]
    view.copy_(_normal(11, 2, 20001, "bf16"))
    _check(wsw, view, [5, 20000], 8, 1.0)
