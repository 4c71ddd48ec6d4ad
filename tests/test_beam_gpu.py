"""Beam selection on the GPU against the double-precision oracle."""
import math

import numpy as np
import pytest
import torch

import oracle
from paged_latent_attention_gb300 import api

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def _check(logits, scores, **kw):
    tokens, parents, best = api.mla_beam_select(logits, scores, **kw)
    ended = kw.get("ended")
    want = oracle.beam_select(logits.double().cpu().numpy(), scores.double().cpu().numpy(),
                              None if ended is None else ended.cpu().numpy(),
                              kw.get("end_token", -1))
    assert tokens.dtype == parents.dtype == torch.int32
    assert np.array_equal(tokens.cpu().numpy(), want[0])
    assert np.array_equal(parents.cpu().numpy(), want[1])
    got = best.double().cpu().numpy()
    inf = np.isneginf(want[2])
    assert np.array_equal(np.isneginf(got), inf)
    # the sums' fp32 terms (exponentials off by 2^-21 of themselves) and one rounding to fp32
    with np.errstate(invalid="ignore"):
        assert np.all(inf | (np.abs(got - want[2]) <= 2.0 ** -21 + 2.0 ** -24 * np.abs(want[2])))


def _inputs(B, K, V, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = (3 * torch.randn(B * K, V, generator=g, device="cuda")).to(dtype)
    scores = torch.randn(B, K, generator=g, device="cuda") - 10
    return logits, scores


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,K,V", [
    (1, 1, 1), (1, 1, 40_000), (3, 2, 2), (1, 4, 5), (2, 4, 32_000), (5, 3, 777), (1, 32, 33),
    (2, 33, 8193), (1, 64, 64), (1, 64, 3), (40, 8, 8192), (7, 5, 20_001), (3, 31, 2048),
    (300, 1, 100), (9, 17, 16_385)])
def test_selection_matches_the_oracle(B, K, V, dtype):
    _check(*_inputs(B, K, V, dtype, 7 * B + K))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,K,V", [(2, 4, 3000), (1, 40, 9000), (60, 3, 20_000)])
@pytest.mark.parametrize("kind", ["equal", "few", "masked", "all masked", "ramp", "heavy thread"])
def test_ties_and_masked_tokens(kind, B, K, V, dtype):
    """Ties go to the lowest beam, then token, however many there are."""
    logits, scores = _inputs(B, K, V, dtype, K)
    scores[:] = -3.0
    if kind == "equal":
        logits.fill_(0.5)
    elif kind == "few":
        logits = (torch.arange(V, device="cuda") * 7919 % 5).to(dtype).repeat(B * K, 1)
    elif kind == "masked":
        logits[:, K // 2:] = -math.inf
    elif kind == "all masked":
        logits[::2] = -math.inf
    elif kind == "ramp":
        logits = (torch.arange(V, device="cuda") / 64).to(dtype).repeat(B * K, 1)
    else:
        logits.fill_(-1.0)
        logits[:, 16:24] = torch.linspace(0, 1, 8, device="cuda").to(dtype)
        logits[:, -3:] = 0.5
    _check(logits.contiguous(), scores)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K,V", [(4, 1000), (32, 20), (40, 25_000), (3, 60_000)])
def test_unused_ended_and_broken_beams(K, V, dtype):
    logits, scores = _inputs(6, K, V, dtype, V)
    scores[0, 1:] = -math.inf                       # the first step of a search
    scores[1] = -math.inf                           # nothing to go on from
    logits[2 * K, 5] = math.nan
    logits[2 * K + 1, 0] = math.inf
    ended = torch.zeros(6, K, dtype=torch.bool, device="cuda")
    ended[3, 0] = ended[3, -1] = True
    ended[4] = True
    ended[0, 0] = True
    scores[5, 2] = math.nan
    _check(logits, scores)
    for end in (0, V - 1, 7):
        _check(logits, scores, ended=ended, end_token=end)
    _check(logits, scores, ended=ended.to(torch.uint8), end_token=3)


def test_a_row_of_nan_everywhere_writes_nothing_else():
    logits, scores = _inputs(2, 64, 70_000, torch.bfloat16, 3)
    logits[5] = math.nan
    logits[9, ::2] = math.nan
    _check(logits, scores)


def test_views_outputs_and_workspace():
    logits, scores = _inputs(2, 3, 501, torch.bfloat16, 1)
    wide = torch.full((6, 777), 9.0, dtype=torch.bfloat16, device="cuda")
    for off in (0, 3, 8):
        view = wide[:, off:off + 501]
        view.copy_(logits)
        _check(view, scores)
    tokens = torch.full((2, 3), -5, dtype=torch.int32, device="cuda")
    work = api.allocate_beam_workspace(2, 3, 501)
    work.fill_(255)
    got = api.mla_beam_select(logits, scores, tokens=tokens, workspace=work)
    assert got[0].data_ptr() == tokens.data_ptr()
    assert torch.equal(tokens, api.mla_beam_select(logits, scores)[0])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,K,V", [(8, 4, 32_000), (10, 5, 20_000), (100, 1, 8000), (1, 64, 9000),
                                   (3, 4, 2048), (2, 8, 2043), (2, 2, 16_384)])
def test_nothing_behind_the_workspace_is_written(B, K, V, dtype):
    """Also where 16-bit rows are cut shorter than fp32 rows of the same length."""
    size = api.allocate_beam_workspace(B, K, V).numel()
    room = torch.full((2 * size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    _check(*_inputs(B, K, V, dtype, K), workspace=room[:size])
    assert bool((room[size:] == 0xA5).all())


def test_other_stream_and_graph_replay():
    logits, scores = _inputs(4, 4, 30_000, torch.float32, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = api.mla_beam_select(logits, scores)
    got = api.mla_beam_select(logits, scores, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = api.mla_beam_select(logits, scores)
    for seed in (5, 6):
        x, s = _inputs(4, 4, 30_000, torch.float32, seed)
        logits.copy_(x)
        scores.copy_(s)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, api.mla_beam_select(x, s)))


def test_refusals():
    logits, scores = _inputs(2, 3, 50, torch.float32, 1)
    flags = torch.zeros(2, 3, dtype=torch.bool, device="cuda")
    bad = [
        lambda: api.mla_beam_select(logits.double(), scores),
        lambda: api.mla_beam_select(logits[:5], scores),
        lambda: api.mla_beam_select(logits.t(), scores),
        lambda: api.mla_beam_select(logits, scores.double()),
        lambda: api.mla_beam_select(logits, scores.cpu()),
        lambda: api.mla_beam_select(logits, scores, out_scores=scores),
        lambda: api.mla_beam_select(logits, scores, ended=flags),
        lambda: api.mla_beam_select(logits, scores, ended=flags, end_token=50),
        lambda: api.mla_beam_select(logits, scores, ended=flags.int(), end_token=0),
        lambda: api.mla_beam_select(logits, scores, tokens=torch.zeros(2, 3, device="cuda")),
        lambda: api.mla_beam_select(logits, scores, workspace=torch.empty(47, device="cuda")),
        lambda: api.mla_beam_select(logits.clone().requires_grad_(), scores),
        lambda: api.mla_beam_select(torch.zeros(65, 9, device="cuda"),
                                    torch.zeros(1, 65, device="cuda")),
    ]
    for call in bad:
        with pytest.raises((ValueError, RuntimeError)):
            call()
