"""The forms of the accumulated weight that run on pairs of CTAs, launched back to back
with forms that lay out the same shared memory differently: what a pair's last commits
signal arrives while both CTAs are still there, so every launch gives the bits that it
gives alone, and no wait gives up."""
import pytest
import torch

from paged_latent_attention_gb300 import api, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
def test_pairs_back_to_back(fp8):
    w = inputs.custom_workload([3000, 1, 700, 0, 260], 1, 16, seed=7)
    slab = (inputs.make_slab_e4m3 if fp8 else inputs.make_slab)(w, "cuda", poison_nan=True)
    ids, lens = (torch.as_tensor(a, device="cuda") for a in (w.page_table, w.seq_lens))
    g = torch.Generator(device="cuda").manual_seed(8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    forms = []
    for n_q, H in ((3, 64), (1, 64), (5, 128), (2, 128), (1, 128), (17, 16), (40, 16)):
        T = w.num_reqs * n_q
        forms.append((n_q, torch.randn(T, H, 512, device="cuda", generator=g).to(torch.bfloat16),
                      torch.randn(T, H, 64, device="cuda", generator=g).to(torch.bfloat16),
                      torch.full((T, H), 9.0, device="cuda")))

    def run(form, mass):
        n_q, qn, qr, lse = form
        args = (qn, qr, lse, slab, ids, lens, mass)
        if fp8:
            api.mla_attention_mass_fp8(*args, n_q=n_q, decay=0.0, status=status,
                                       kv_scale=inputs.KV_SCALE_E4M3)
        else:
            api.mla_attention_mass(*args, n_q=n_q, decay=0.0, status=status)
        return mass

    want = []
    for form in forms:
        want.append(run(form, torch.zeros(w.num_reqs, 3000, device="cuda")))
        torch.cuda.synchronize()
    got = [[run(form, torch.zeros_like(want[0])) for form in forms] for _ in range(20)]
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for row in got:
        assert all(torch.equal(a, b) for a, b in zip(row, want))
