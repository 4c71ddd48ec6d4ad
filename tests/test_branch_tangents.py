"""Derivatives that the operators for continuations would lose, in forward mode (CPU only)."""
import pytest
import torch
from torch.autograd import forward_ad

from paged_latent_attention_gb300 import api


def test_tangents_are_not_lost_without_a_word():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    x = torch.zeros(2, 4, 512, dtype=torch.bfloat16)
    slab = torch.zeros(1, 1536 * 576, dtype=torch.bfloat16)
    logits, scores = torch.zeros(4, 9), torch.zeros(2, 2)
    with forward_ad.dual_level():
        dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))
        for k in range(4):
            args = [x, x[..., :64], x, slab]
            args[k] = dual(args[k])
            with pytest.raises(ValueError, match="tangents"):
                api.mla_decode_shared(*args, i(2, 3), i(2), i(2), i(1))
        for a, b in ((dual(logits), scores), (logits, dual(scores))):
            with pytest.raises(ValueError, match="tangents"):
                api.mla_beam_select(a, b)
        # without them it is the device that is asked for
        with pytest.raises(ValueError, match="CUDA"):
            api.mla_beam_select(logits, scores)
    with pytest.raises(ValueError, match="autograd"):
        api.mla_beam_select(logits.requires_grad_(), scores)
