"""The loop that holds a cache to a budget, through more than one eviction: append,
decode, accumulate, select, compact, and on from there with what the calls returned."""
import math

import numpy as np
import pytest
import torch

import oracle
from helpers import SCALE, assert_parity
from paged_latent_attention_gb300 import api, inputs

pytestmark = pytest.mark.gpu

PT = inputs.PAGE_TOKENS


def _dirty(*shape):
    """Leaves NaN where the allocator's next tensor of this size will lie."""
    x = torch.full(shape, math.nan, device="cuda")
    torch.cuda.synchronize()
    del x


def _ints(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32), device="cuda")


def test_evictions_one_after_another():
    """Appends, decodes and accumulations, three times over with an eviction after each.
    Every step adds its H rows' weights (the decode's lse is within 1e-3: a row's
    weights sum to 1 within e^(2e-3) - 1), the tokens appended since an eviction
    among them; each eviction keeps the newest tokens; one history stays below the
    budget throughout."""
    R, H, keep, recent, room = 3, 16, 1532, 8, 2100
    g = torch.Generator().manual_seed(3)
    lens = np.array([1990, 700, 1700])
    at = lens.copy()                                   # the next tokens' positions
    w = inputs.custom_workload([int(v) + 8 for v in lens], 1, H, seed=5, spare_pages=20)
    slab = inputs.make_slab(w, "cuda", poison_nan=False)
    table = api.rope_table(64, base=50000.0)
    ids = torch.as_tensor(w.page_table, device="cuda")
    free = [p for p in range(w.num_pages) if p not in set(w.page_table.reshape(-1).tolist())]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mass = torch.zeros(R, room, device="cuda")
    for cycle in range(3):
        for _ in range(6):
            lens = lens + 1
            rows = [torch.randn(R, d, generator=g).to(torch.bfloat16).cuda() for d in (512, 64)]
            q = torch.randn(R, H, 576, generator=g).to(torch.bfloat16).cuda()
            qr = api.mla_kv_append_rope(*rows, slab, ids, _ints(lens), 1, table,
                                        positions=_ints(at), q_rope=q[..., 512:], status=status)
            at = at + 1
            qn = q[..., :512].contiguous()
            gate = torch.randn(R, H, 512, generator=g).to(torch.bfloat16)
            out, lse = api.mla_decode(qn, qr, gate.cuda(), slab, ids, _ints(lens))
            before = mass.double().sum(1).cpu().numpy()
            api.mla_attention_mass(qn, qr, lse, slab, ids, _ints(lens), mass, status=status)
            total = mass.double().sum(1).cpu().numpy()
            assert np.all(np.isfinite(total))
            # (the stored sums round by 2^-24 each)
            slack = (math.exp(2e-3) - 1) * H + 2.0 ** -23 * total
            assert np.all(np.abs(total - before - H) <= slack)
            for r in range(R):
                assert bool((mass[r, : lens[r]] > 0).all()) and bool((mass[r, lens[r]:] == 0).all())
        ref_out, ref_lse = oracle.mla_decode_reference(
            qn.cpu(), qr.cpu(), gate, slab.cpu(), ids.cpu().numpy(), lens.astype(np.int32), 1, H,
            SCALE, num_pages=w.num_pages)
        assert_parity(out, lse, ref_out, ref_lse, what=f"decode after {cycle} evictions")

        kept, n = api.mla_evict_select(mass, _ints(lens), keep, sink=4, recent=recent,
                                       status=status)
        want = oracle.evict_select(mass.cpu().numpy(), lens, keep, 4, recent)
        assert [kept[r, : len(k)].tolist() for r, k in enumerate(want)] == want
        for r, k in enumerate(want):
            assert k[-recent:] == list(range(lens[r] - recent, lens[r]))
        cols = -(-(keep + 8) // PT)
        fresh = torch.tensor([[free.pop() for _ in range(cols)] for _ in range(R)],
                             dtype=torch.int32, device="cuda")
        _dirty(R, room)
        _dirty(R, kept.shape[1])
        carried = api.mla_kv_compact([slab], ids, _ints(lens), fresh, kept, n, mass=mass,
                                     status=status)
        for r, k in enumerate(want):
            assert torch.equal(carried[r, : len(k)], mass[r, torch.tensor(k).cuda()])
        mass, ids, lens = carried, fresh, np.array([len(k) for k in want])
        assert n.tolist() == lens.tolist() and mass.shape[1] >= room
        for r in range(R):
            assert bool((mass[r, lens[r]:] == 0).all())
    assert int(status.item()) == 0 and lens[1] < keep and lens[0] == lens[2] == keep
