"""Calls of the cache-budget operators on streams of their own, with the memory that
they allocate by default, behind work that is still queued on the caller's stream."""
import pytest
import torch

from paged_latent_attention_gb300 import api, inputs

pytestmark = pytest.mark.gpu

PT, ROW = inputs.PAGE_TOKENS, inputs.ROW_ELEMS


def _freed(shape, dtype):
    """Address of a block that the current stream has just given back."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    at = t.data_ptr()
    del t
    return at


def test_outputs_are_not_the_callers_freed_blocks():
    side = torch.cuda.Stream()
    table, pos = api.rope_table(64), torch.arange(700, dtype=torch.int32, device="cuda")
    x = torch.randn(700, 5, 64, device="cuda")
    mass = torch.rand(3, 5000, device="cuda")
    lens = torch.tensor([5000, 4000, 10], dtype=torch.int32, device="cuda")
    slab = torch.zeros(6, PT * ROW, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    fresh = torch.tensor([[3], [4], [5]], dtype=torch.int32, device="cuda")
    want, n = api.mla_evict_select(mass, lens, 900, recent=5)
    turned = api.mla_rope(x, pos, table)
    carried = api.mla_kv_compact([slab], ids, lens, fresh, want, n, mass=mass)
    torch.cuda.synchronize()

    at = _freed(x.shape, x.dtype)
    got = api.mla_rope(x, pos, table, stream=side)
    assert got.data_ptr() != at
    at = _freed(want.shape, want.dtype)
    kept, m = api.mla_evict_select(mass, lens, 900, recent=5, stream=side)
    assert kept.data_ptr() != at
    at = _freed(carried.shape, carried.dtype)
    out = api.mla_kv_compact([slab], ids, lens, fresh, want, n, mass=mass, stream=side)
    assert out.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(got, turned) and torch.equal(out, carried) and torch.equal(m, n)
    assert all(torch.equal(kept[r, : n[r]], want[r, : n[r]]) for r in range(3))


def test_default_workspaces_of_two_streams():
    """A call that waits on the caller's stream, and one on another stream right after it:
    each keeps the split queries (mass) and histograms (selection) of its own."""
    w = inputs.custom_workload([3000, 2000], 4, 64, seed=2)
    slab = inputs.make_slab_e4m3(w, "cuda", poison_nan=False)
    ids, lens = (torch.as_tensor(a, device="cuda") for a in (w.page_table, w.seq_lens))
    g = torch.Generator(device="cuda").manual_seed(4)
    steps = [(torch.randn(8, 64, 512, device="cuda", generator=g).to(torch.bfloat16),
              torch.randn(8, 64, 64, device="cuda", generator=g).to(torch.bfloat16),
              torch.full((8, 64), 9.0, device="cuda")) for _ in range(2)]
    rows = [torch.rand(2, 500_000, device="cuda", generator=g) for _ in range(2)]
    long = torch.tensor([500_000, 400_001], dtype=torch.int32, device="cuda")

    def calls(i, mass, stream=None):
        api.mla_attention_mass_fp8(*steps[i], slab, ids, lens, mass, n_q=4,
                                   kv_scale=inputs.KV_SCALE_E4M3, stream=stream)
        return api.mla_evict_select(rows[i], long, 40_000, sink=4, recent=99, stream=stream)

    wanted = []
    for i in range(2):
        mass = torch.zeros(2, 3000, device="cuda")
        wanted.append((mass, *calls(i, mass)))
    sums = [torch.zeros(2, 3000, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                     # some 10 ms on the caller's stream
    first = calls(0, sums[0])
    second = calls(1, sums[1], side)
    torch.cuda.synchronize()
    for i, got in enumerate(((sums[0], *first), (sums[1], *second))):
        assert all(torch.equal(a, b) for a, b in zip(got, wanted[i])), i
