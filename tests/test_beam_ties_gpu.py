"""Beams that are the same: the same logits and scores, wherever their rows lie in memory."""
import numpy as np
import pytest
import torch

import oracle
from paged_latent_attention_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("B,K,V,seed", [(3, 4, 32_001, 1), (2, 8, 50_003, 2), (1, 64, 4097, 3), (1, 33, 20_001, 4),
                                        (5, 5, 1003, 5), (2, 32, 150_001, 6)])
def test_beams_that_are_the_same_come_in_their_order(B, K, V, seed, dtype):
    """(Rows of an odd length start at every address within a group of 16 bytes.)"""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (2.0 * torch.randn(B, 1, V, generator=g, device="cuda")).to(dtype).repeat(1, K, 1)
    scores = torch.randn(B, 1, generator=g, device="cuda").repeat(1, K).contiguous()
    if K > 4:
        # some are others, in between
        x[:, 1::3] = (2.0 * torch.randn(B, 1, V, generator=g, device="cuda")).to(dtype)
        scores[:, 2::5] -= 0.25
    x = x.view(B * K, V).contiguous()
    tokens, parents, best = api.mla_beam_select(x, scores)
    want = oracle.beam_select(x.double().cpu().numpy(), scores.double().cpu().numpy())
    assert np.array_equal(tokens.cpu().numpy(), want[0])
    assert np.array_equal(parents.cpu().numpy(), want[1])
    assert np.abs(best.double().cpu().numpy() - want[2]).max() <= 3e-6 + 2.0 ** -24 * np.abs(want[2]).max()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("V", [1003, 20_001])
def test_beams_with_the_same_logits_at_other_tokens_tie(V, dtype):
    """The same logits in another order: the same log-sum-exp."""
    g = torch.Generator(device="cuda").manual_seed(V)
    K = 6
    row = (2.0 * torch.randn(V, generator=g, device="cuda")).to(dtype)
    x = torch.stack([row[torch.randperm(V, generator=g, device="cuda")] for _ in range(K)])
    tokens, parents, _ = api.mla_beam_select(x, torch.full((1, K), -1.5, device="cuda"))
    flat = x.double().view(-1).cpu().numpy()
    want = np.lexsort((np.arange(flat.size), -flat))[:K]
    assert tokens[0].tolist() == (want % V).tolist() and parents[0].tolist() == (want // V).tolist()


@pytest.mark.parametrize("V", [2001, 50_001])
def test_beams_that_are_almost_the_same_stay_apart(V):
    """Nearly equal logits with the same largest, log-sum-exps some 1e-6 apart: each beam
    has its own (within the bound for any row, less than their distance)."""
    g = torch.Generator(device="cuda").manual_seed(V)
    K = 8
    x = (0.01 * torch.randn(V, generator=g, device="cuda")).repeat(K, 1)
    x[:, 7] = 0.5
    x[:, 11] = torch.log(1.0 + 0.7e-6 * V * torch.arange(K, device="cuda"))
    assert float(x[:, 11].max()) < 0.5
    lse = torch.logsumexp(x.double(), 1)
    scores = (lse - 0.5).float()[None].contiguous()
    _, parents, best = api.mla_beam_select(x, scores)
    want = scores.double()[0] + 0.5 - lse
    got = best.double()[0]
    assert bool(((got - want[parents[0].long()]).abs() <= 1.5e-6).all())
