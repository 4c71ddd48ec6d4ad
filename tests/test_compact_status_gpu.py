"""Kept tokens without a weight are reported by the compaction."""
import pytest
import torch

from paged_latent_attention_gb300 import api, inputs

pytestmark = pytest.mark.gpu

PT, ROW = inputs.PAGE_TOKENS, inputs.ROW_ELEMS


@pytest.mark.parametrize("fp8", [False, True])
def test_kept_tokens_past_the_weights(fp8):
    """Rows of 900 weights for histories of 1,000 and 800 tokens: the rows of all kept
    tokens are copied, those from 900 on without a weight, which the status word says."""
    slab = torch.randint(0, 255, (4, PT * ROW * (1 if fp8 else 2)), dtype=torch.uint8,
                         device="cuda")
    slab = slab if fp8 else slab.view(torch.bfloat16)
    ids = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    fresh = torch.tensor([[2], [3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([1000, 800], dtype=torch.int32, device="cuda")
    mass = torch.rand(2, 900, device="cuda") + 1.0
    kept = torch.stack([torch.arange(700) + 250, torch.arange(700) + 100]).to(torch.int32).cuda()
    for counts, code in (([700, 700], 34), ([650, 700], 0)):
        n = torch.tensor(counts, dtype=torch.int32, device="cuda")
        pool, status = slab.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
        out = api.mla_kv_compact([pool], ids, lens, fresh, kept, n, mass=mass, status=status)
        assert int(status.item()) == code
        assert torch.equal(out[0, :650], mass[0, 250:900]) and bool((out[0, 650:] == 0).all())
        assert torch.equal(out[1, :700], mass[1, 100:800]) and bool((out[1, 700:] == 0).all())
        rows = pool.view(torch.uint8).view(4, PT, -1)
        for r, first in enumerate((250, 100)):
            assert torch.equal(rows[2 + r, : counts[r]], rows[r, first:first + counts[r]])
