"""Page tables that are views of wider buffers, used past the view's columns: what the
neighbouring columns hold (here the IDs of live pages of the pool) is not part of the
table, so such tokens are reported with 33, nothing is read or written through those
columns, and everything inside the view comes out as from a table of its own."""
import numpy as np
import pytest
import torch

from paged_latent_attention_gb300 import api, inputs

pytestmark = pytest.mark.gpu

PT, ROW = inputs.PAGE_TOKENS, inputs.ROW_ELEMS


def _setup(fp8, seed):
    """Two histories of three pages, and their table with only two columns in view."""
    w = inputs.custom_workload([4000, 3500], 1, 16, seed=seed, spare_pages=6)
    slab = (inputs.make_slab_e4m3 if fp8 else inputs.make_slab)(w, "cuda", poison_nan=False)
    full = torch.as_tensor(w.page_table, device="cuda").contiguous()
    assert full.shape == (2, 3) and bool((full >= 0).all())
    lens = torch.as_tensor(w.seq_lens, device="cuda")
    free = [p for p in range(w.num_pages) if p not in set(w.page_table.reshape(-1).tolist())]
    return w, slab, full, full[:, :2], lens, free


def _bits(slab):
    return slab.view(torch.uint8)


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fp8", [False, True])
def test_append_past_the_view(fp8):
    w, slab, full, view, _, _ = _setup(fp8, 1)
    g = torch.Generator().manual_seed(1)
    # four new tokens each: request 0 passes the view's last row by two, request 1 ends inside
    lens = torch.tensor([2 * PT + 2, 2 * PT - 5], dtype=torch.int32, device="cuda")
    lat, rope = (torch.randn(8, d, generator=g).to(torch.bfloat16).cuda() for d in (512, 64))
    q = torch.randn(8, 3, 64, generator=g).to(torch.bfloat16).cuda()
    table = api.rope_table(64)

    def run(ids):
        pool, status = slab.clone(), _status()
        args = (lat, rope, pool, ids, lens, 4, table)
        if fp8:
            out = api.mla_kv_append_rope_fp8(*args, kv_scale=0.05, q_rope=q, status=status)
        else:
            out = api.mla_kv_append_rope(*args, q_rope=q, status=status)
        return out, pool, int(status.item())

    want, pool, code = run(view.contiguous())
    assert code == 33
    got, seen, code = run(view)
    assert code == 33 and torch.equal(_bits(seen), _bits(pool)) and torch.equal(got, want)
    for r in range(2):
        assert torch.equal(_bits(seen)[full[r, 2]], _bits(slab)[full[r, 2]])


@pytest.mark.parametrize("n_q,H", [(1, 16), (2, 128), (3, 128)])
@pytest.mark.parametrize("fp8", [False, True])
def test_mass_past_the_view(fp8, n_q, H):
    w, slab, full, view, lens, _ = _setup(fp8, 2)
    g = torch.Generator().manual_seed(2)
    qn = torch.randn(2 * n_q, H, 512, generator=g).to(torch.bfloat16).cuda()
    qr = torch.randn(2 * n_q, H, 64, generator=g).to(torch.bfloat16).cuda()
    lse = torch.full((2 * n_q, H), 9.0, device="cuda")

    def run(ids):
        mass, status = torch.ones(2, 4100, device="cuda"), _status()
        args = (qn, qr, lse, slab, ids, lens, mass)
        if fp8:
            api.mla_attention_mass_fp8(*args, kv_scale=inputs.KV_SCALE_E4M3, n_q=n_q, status=status)
        else:
            api.mla_attention_mass(*args, n_q=n_q, status=status)
        return mass, int(status.item())

    whole, code = run(full)
    assert code == 0
    mass, code = run(view)
    assert code == 33
    assert torch.equal(mass[:, : 2 * PT], whole[:, : 2 * PT])
    assert bool((mass[:, 2 * PT:] == 1).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_compaction_past_the_views(fp8):
    w, slab, full, view, lens, free = _setup(fp8, 3)
    kept = torch.stack([torch.arange(1600), torch.arange(1600) + 1800]).to(torch.int32).cuda()
    n = torch.full((2,), 1600, dtype=torch.int32, device="cuda")
    fresh = torch.tensor([free[:2], free[2:4]], dtype=torch.int32, device="cuda")

    def run(ids, outs):
        pool, status = slab.clone(), _status()
        api.mla_kv_compact([pool], ids, lens, outs, kept, n, status=status)
        return _bits(pool), int(status.item())

    whole, code = run(full, fresh)
    assert code == 0
    # new histories of 1,600 rows with one page each in view
    pool, code = run(full, fresh[:, :1])
    assert code == 33
    for r in range(2):
        assert torch.equal(pool[fresh[r, 0]], whole[fresh[r, 0]])
        assert torch.equal(pool[fresh[r, 1]], _bits(slab)[fresh[r, 1]])
    # old histories: request 1's tokens past its second page lie past the view
    pool, code = run(view, fresh)
    assert code == 33
    assert torch.equal(pool[fresh[0]], whole[fresh[0]])
    inside, width = 2 * PT - 1800, ROW * (1 if fp8 else 2)
    assert torch.equal(pool[fresh[1, 0], : inside * width], whole[fresh[1, 0], : inside * width])
    assert torch.equal(pool[fresh[1, 0], inside * width:],
                       _bits(slab)[fresh[1, 0], inside * width:])
    assert torch.equal(pool[fresh[1, 1]], _bits(slab)[fresh[1, 1]])
