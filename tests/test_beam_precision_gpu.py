"""The log-sum-exps of beam selection against 64 bits, where the roundings of many equal terms
add up.

A slice's terms are 2^p', p' = 8 - (high - x) log2 e: the rounding of p' (twice in fp32), that of
log2 e (2^-26 of it), 2^-22 for the exponential (what the instruction is documented to do).  They are
added in a tree of six roundings, then in fixed point, and rounded once; a slice whose largest
logit is not the row's is scaled by an exponential (2^-23 and its correction's 2^-24, a
product without loss).  The logarithm is off by 2^-25.  Scores are rounded to fp32, 2^-24 of
themselves.  Half a step of p' is 2^-22 down to p' = -8 and 2^-21 to -16, so with up to a few
million logits a log-sum-exp is off by less than
  2^-22 + 2 ln 2 2^-21 / 2 + 16.6 2^-26 + 6 2^-24 + 2^-24 + 3 2^-24 + 2^-25 < 1.5e-6."""
import math

import numpy as np
import pytest
import torch

import oracle
from paged_latent_attention_gb300 import api

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
U = 2.0 ** -24
ANY = 1.5e-6


def _check(logits, scores, tol, choose=True):
    tokens, parents, best = api.mla_beam_select(logits, scores)
    want = oracle.beam_select(logits.double().cpu().numpy(), scores.double().cpu().numpy())
    if choose:
        assert np.array_equal(tokens.cpu().numpy(), want[0])
        assert np.array_equal(parents.cpu().numpy(), want[1])
    err = np.abs(best.double().cpu().numpy() - want[2])
    lim = tol + U * np.abs(want[2])
    assert np.all(err <= lim), (float(err.max()), float((err / lim).max()))


def _level(x):
    """Scores that bring each row's best candidate next to 0, where fp32 is fine."""
    return (torch.logsumexp(x.double(), 1) - x.double().amax(1)).float()[:, None]


def _two_values(x):
    """The bound for rows of two values: the larger one's terms are exact, the smaller one's
    all off by the same."""
    x = x.double()
    high, low = x.amax(1), x.amin(1)
    gap = high - low
    share = (x < high[:, None]).sum(1) * torch.exp(low - torch.logsumexp(x, 1))
    p = (8.0 - gap / math.log(2.0)).abs().clamp(min=1.0)
    half = 2.0 ** (torch.floor(torch.log2(p)) - 24.0)
    tol = share * (2.0 ** -22 + 2 * math.log(2.0) * half + gap * 2.0 ** -26) + 10.5 * U
    return tol.cpu().numpy()[:, None]


def _peaked(peak, rest, V, dtype=torch.float32):
    x = torch.full((1, V), rest, dtype=dtype, device="cuda")
    x[0, V // 3] = peak
    return x


ROWS = [(5.626445, -5.4734426), (2.0329037, -6.0134034)]


@pytest.mark.parametrize("peak,rest", ROWS + [(11.3, 0.1), (0.7, -11.3), (3.3, -1.7), (-20.1, -31.9)])
@pytest.mark.parametrize("V", [8001, 150_001, 1_000_003])
def test_many_equal_logits_below_one(peak, rest, V):
    x = _peaked(peak, rest, V)
    _check(x, _level(x), _two_values(x))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V,every", [(4000, 4000), (8001, 8001), (16_380, 16_380), (20_000, 10_000),
                                     (150_001, 8000)])
def test_many_equal_logits_of_any_value(V, every, dtype):
    """(Rounded in every way that there is.)"""
    g = torch.Generator().manual_seed(1)
    n = 400 if V < 100_000 else 60
    gap = torch.rand(n, generator=g) * 14.0
    high = torch.randn(n, generator=g) * 4.0
    x = (high - gap)[:, None].to(dtype).repeat(1, V)
    x[:, ::every] = high.to(dtype)[:, None]
    x = x.cuda()
    _check(x, _level(x), _two_values(x))


@pytest.mark.parametrize("least", [1.4e-6, -1.4e-6, 3e-6, -3e-6])
def test_beams_that_differ_by_little_come_in_order(least):
    """Rows whose small terms are all rounded up, and all down, beside the large one."""
    x = torch.cat([_peaked(*r, 16_380, torch.bfloat16) for r in
                   ((0.06884765625, -13.625), (-1.1640625, -14.1875))])
    assert float(_two_values(x).sum()) < 1.35e-6
    top = (x.double().amax(1) - torch.logsumexp(x.double(), 1)).tolist()
    # scores below 1, so that a step of them is less than a tenth of the difference
    scores = torch.tensor([[-0.2, -0.2 + top[0] - top[1] + least]], dtype=torch.float32,
                          device="cuda")
    assert abs(float(scores[0, 1])) < 1.0
    _check(x, scores, ANY)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shift", [0.0, 57.0, 61.0, -57.0, -61.0, -64.0, 300.0, -300.0, 20_000.0])
def test_logits_far_from_zero(shift, dtype):
    g = torch.Generator(device="cuda").manual_seed(7)
    x = 2.0 * torch.randn(6, 90_001, generator=g, device="cuda")
    x[:3] -= torch.linspace(0, 30, 90_001, device="cuda")     # slices of falling height
    x[3, 40_000:] = -torch.inf
    x = (x + shift).to(dtype)
    _check(x, torch.zeros(2, 3, device="cuda"), ANY, choose=False)


@pytest.mark.parametrize("dtype", TYPES)
def test_tokens_masked_by_the_lowest_value(dtype):
    lowest = torch.finfo(dtype).min
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(6, 40_001, generator=g, device="cuda").to(dtype)
    x[:, 5:] = lowest
    scores = torch.randn(2, 3, generator=g, device="cuda")
    _check(x, scores, ANY)
    x[1, 7] = -torch.inf
    x[:, 20_000:] = -torch.inf
    _check(x, scores, ANY)
    # rows of nothing else, where 64 bits would lose ln V beside the logits: score - ln V
    for value in (lowest, torch.finfo(dtype).max):
        x[:, :20_000] = value
        tokens, parents, best = api.mla_beam_select(x, scores)
        assert tokens.tolist() == [[0, 1, 2]] * 2
        want, k = scores.double().max(1)
        assert torch.equal(parents.long(), (k + torch.tensor([0, 3], device="cuda"))[:, None].expand(2, 3))
        err = (best.double() - (want - math.log(20_000.0))[:, None]).abs()
        assert bool((err <= ANY + U * 13.0).all())
