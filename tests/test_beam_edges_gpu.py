"""Beam selection at the ends of what it takes."""
import math

import pytest
import torch

from paged_latent_attention_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("off", [1, 7])
def test_the_largest_vocabulary_at_any_address(off, dtype):
    """2^31 - 1 tokens in a row that starts inside a group of 16 bytes: the first slice counts."""
    V = 2 ** 31 - 1
    x = torch.zeros(V + off, dtype=dtype, device="cuda")[off:].view(1, V)
    peaks = {0: 15.0, 100: 14.0, 2000: 13.0, V - 1: 12.0}
    for v, h in peaks.items():
        x[0, v] = h
    total = math.log(V - len(peaks) + sum(math.exp(h) for h in peaks.values()))
    scores = torch.zeros(1, 1, device="cuda")
    for v, h in peaks.items():
        tokens, parents, best = api.mla_beam_select(x, scores)
        assert tokens.tolist() == [[v]] and parents.tolist() == [[0]]
        assert abs(float(best) - (h - total)) <= 2.0 ** -21 + 2.0 ** -24 * abs(h - total)
        x[0, v] = 0.0
        total = math.log(math.exp(total) - math.exp(h) + 1.0)
