"""Outputs beside their inputs in one buffer: accepted, and nothing else is written."""
import pytest
import torch

from paged_latent_attention_gb300 import api, inputs

pytestmark = pytest.mark.gpu

PT, ROW = inputs.PAGE_TOKENS, inputs.ROW_ELEMS


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rotated_part_beside_its_input(layout, dtype):
    g = torch.Generator().manual_seed(2)
    wide = torch.randn(37, 5, 160, generator=g).to(dtype).cuda()
    before = wide.clone()
    pos = torch.arange(37, dtype=torch.int32, device="cuda") * 1000
    table = api.rope_table(64)
    want = api.mla_rope(before[..., :64], pos, table, layout=layout)
    api.mla_rope(wide[..., :64], pos, table, layout=layout, out=wide[..., 64:128])
    assert torch.equal(wide[..., 64:128], want)
    assert torch.equal(wide[..., :64], before[..., :64])
    assert torch.equal(wide[..., 128:], before[..., 128:])
    for bad in (wide[..., 63:127], wide[..., 1:65]):
        with pytest.raises(ValueError):
            api.mla_rope(wide[..., :64], pos, table, layout=layout, out=bad)


def test_carried_weights_beside_the_weights():
    slab = torch.zeros(4, PT * ROW, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([1000, 800], dtype=torch.int32, device="cuda")
    both = torch.rand(2, 1700, device="cuda")
    before = both.clone()
    kept, n = api.mla_evict_select(both[:, :1000], lens, 600, recent=7)
    api.mla_kv_compact([slab], ids, lens, ids + 2, kept, n, mass=both[:, :1000],
                       mass_out=both[:, 1000:])
    assert torch.equal(both[:, 1000:1600], before.gather(1, kept.long()))
    assert torch.equal(both[:, :1000], before[:, :1000])
    assert torch.equal(both[:, 1600:], before[:, 1600:])
    with pytest.raises(ValueError):
        api.mla_kv_compact([slab], ids, lens, ids + 2, kept, n, mass=both[:, :1000],
                           mass_out=both[:, 999:])
