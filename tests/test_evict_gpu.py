"""Eviction selection and page compaction on the GPU: exact against the oracle, and
a run of the operators together as a server uses them."""
import math

import numpy as np
import pytest
import torch

import oracle
from helpers import SCALE, assert_parity
from paged_latent_attention_gb300 import _native, api, inputs

pytestmark = pytest.mark.gpu

PT, ROW = inputs.PAGE_TOKENS, inputs.ROW_ELEMS


def _select(mass, lens, keep, sink, recent, **kw):
    R = mass.shape[0]
    cols = min(keep, mass.shape[1])
    kept = torch.full((R, cols + 3), -7, dtype=torch.int32, device="cuda")
    kept, n = api.mla_evict_select(mass, torch.as_tensor(np.asarray(lens, dtype=np.int32),
                                                         device="cuda"),
                                   keep, sink=sink, recent=recent, kept=kept, **kw)
    return kept.cpu().numpy(), n.cpu().numpy()


def _check_select(mass, lens, keep, sink, recent):
    kept, n = _select(mass, lens, keep, sink, recent)
    want = oracle.evict_select(mass.cpu().numpy(), lens, keep, sink, recent)
    for r, rows in enumerate(want):
        assert int(n[r]) == len(rows)
        assert kept[r, : len(rows)].tolist() == rows, r
        assert np.all(kept[r, len(rows):] == -7), "entries past the count were written"


@pytest.mark.parametrize("lengths,keep,sink,recent", [
    ([1], 1, 0, 0), ([0, 1, 2, 3], 2, 1, 1), ([1000, 2000], 512, 4, 64), ([33, 32, 31], 32, 0, 0),
    ([5000, 12, 4097], 700, 0, 0), ([5000, 12, 4097], 700, 350, 350), ([5000, 4097], 1, 0, 0),
    ([9000, 20_000, 0], 8999, 17, 101), ([40_000, 33_000, 90_001], 20_000, 4, 1000),
    ([7] * 300, 3, 1, 1), ([6000] * 90, 100, 2, 30), ([400_000], 60_000, 4, 512),
    ([300_000, 7, 299_999], 500, 3, 5), ([1_000_003], 1, 0, 0), ([270_000, 270_001], 270_000, 1, 9)])
def test_selection_matches_the_oracle(lengths, keep, sink, recent):
    g = torch.Generator().manual_seed(len(lengths) + keep)
    mass = torch.empty(len(lengths), max(max(lengths), 1)).exponential_(generator=g).pow_(3).cuda()
    _check_select(mass, lengths, keep, sink, recent)


@pytest.mark.parametrize("kind", ["equal", "few", "signs", "special", "nan", "tiny"])
@pytest.mark.parametrize("L,keep", [(3000, 1000), (70_000, 30_001), (280_000, 100_003)])
def test_ties_signs_and_special_values(kind, L, keep):
    g = torch.Generator().manual_seed(L)
    m = torch.randn(2, L, generator=g)
    if kind == "equal":
        m.fill_(0.25)
    elif kind == "few":
        m = torch.randint(0, 3, (2, L), generator=g).float()
    elif kind == "signs":
        m = torch.where(torch.randint(0, 2, (2, L), generator=g) > 0, 0.0, -0.0)
        m[:, ::7] = -1.0
    elif kind == "special":
        for i, v in enumerate((math.inf, -math.inf, math.nan, torch.finfo(torch.float32).min,
                               torch.finfo(torch.float32).max, 1e-45, -1e-45)):
            m[:, i::11] = v
    elif kind == "nan":
        m.fill_(math.nan)
        m[:, 5::1000] = -math.inf
    else:
        m = m * 1e-42                      # subnormal weights
    _check_select(m.cuda(), [L, L - 1], keep, 2, 3)


def test_long_rows_with_and_without_a_workspace():
    """The form for long rows takes a workspace; without one (through the C entry) the
    cluster form gives the same indices, and too small a one is refused."""
    g = torch.Generator().manual_seed(1)
    R, L, keep = 2, 500_001, 40_000
    mass = torch.randint(0, 50_000, (R, L), generator=g).float().cuda()
    lens = torch.tensor([L, 300_000], dtype=torch.int32, device="cuda")
    size = _native.lib().mla_evict_workspace_size(R, L)
    assert size > 0 and api.allocate_evict_workspace(R, 2000).numel() == 0
    want, n = api.mla_evict_select(mass, lens, keep, sink=4, recent=100)
    dirty = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        got, m = api.mla_evict_select(mass, lens, keep, sink=4, recent=100, workspace=dirty)
        assert torch.equal(got, want) and torch.equal(m, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.mla_evict_select(mass, lens, keep, sink=4, recent=100, kept=got, kept_lens=m,
                             workspace=dirty)
    lens.copy_(torch.tensor([keep, 400_001], dtype=torch.int32))   # a row without a choice
    mass.copy_(mass.flip(1))
    graph.replay()
    want = oracle.evict_select(mass.cpu().numpy(), lens.tolist(), keep, 4, 100)
    assert [got[r].tolist() for r in range(R)] == want and m.tolist() == [keep, keep]
    want = torch.tensor(want, dtype=torch.int32, device="cuda")
    got.fill_(-1)
    call = (mass.data_ptr(), L, L, lens.data_ptr(), R, keep, 4, 100, got.data_ptr(), keep,
            m.data_ptr())
    assert _native.lib().mla_evict_select(*call, None, 0, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert _native.lib().mla_evict_select(*call, dirty.data_ptr(), size // 2, None) == 3


def test_selection_views_bits_and_graphs():
    g = torch.Generator().manual_seed(3)
    holder = torch.rand(5, 9000, generator=g).cuda()
    lens = [8000, 10, 7999, 4000, 0]
    view = holder[:, 500:8500]
    _check_select(view, lens, 1234, 5, 60)
    # a history longer than its row of weights is taken as the row's length
    _check_select(holder[:, :3000], lens, 100, 1, 1)
    dev = torch.as_tensor(np.asarray(lens, dtype=np.int32), device="cuda")
    want, n = api.mla_evict_select(view, dev, 1234, sink=5, recent=60)
    kept, m = torch.empty_like(want), torch.empty_like(n)
    api.mla_evict_select(view, dev, 1234, sink=5, recent=60, kept=kept, kept_lens=m)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.mla_evict_select(view, dev, 1234, sink=5, recent=60, kept=kept, kept_lens=m)
    kept.fill_(-1)
    holder.copy_(torch.rand(5, 9000, generator=g))
    graph.replay()
    torch.cuda.synchronize()
    for r, rows in enumerate(oracle.evict_select(view.cpu().numpy(), lens, 1234, 5, 60)):
        assert kept[r, : len(rows)].tolist() == rows and int(m[r]) == len(rows)


def _pool(w, fp8, extra, seed=0):
    """Random bits everywhere (NaN among them): the copy must not interpret them."""
    rng = np.random.Generator(np.random.PCG64(seed + 50))
    kind = np.uint8 if fp8 else np.uint16
    bits = rng.integers(0, np.iinfo(kind).max, (w.num_pages + extra, w.page_stride), dtype=kind,
                        endpoint=True)
    return bits


def _fresh(w, counts, extra):
    table = np.zeros((w.num_reqs, max(1, max(-(-c // PT) for c in counts))), dtype=np.int32)
    ids = np.random.Generator(np.random.PCG64(8)).permutation(extra) + w.num_pages
    at = 0
    for r, c in enumerate(counts):
        k = -(-c // PT)
        table[r, :k] = ids[at:at + k]
        at += k
    return table


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lengths,keep,layers,pad", [
    ([5], 1, 1, 0), ([2000, 4000, 0, 1536], 1537, 2, 0), ([3100, 700], 700, 3, 32),
    ([200] * 40, 77, 1, 0), ([1600], 1600, 70, 0)])
def test_compaction_is_exact(fp8, lengths, keep, layers, pad):
    w = inputs.custom_workload(lengths, 1, 16, seed=len(lengths), page_stride=PT * ROW + pad)
    rng = np.random.Generator(np.random.PCG64(2))
    kept = [sorted(rng.choice(L, size=min(L, keep), replace=False).tolist()) for L in lengths]
    extra = sum(-(-len(k) // PT) for k in kept) + 1
    out_table = _fresh(w, [len(k) for k in kept], extra)
    pools = [_pool(w, fp8, extra, l) for l in range(min(layers, 3))]
    dev = [torch.from_numpy(pools[l % len(pools)].view(np.uint8 if fp8 else np.int16)).cuda()
           for l in range(layers)]
    dev = [x if fp8 else x.view(torch.bfloat16) for x in dev]
    idx = np.full((len(lengths), keep + 2), 2**31 - 1, dtype=np.int32)
    for r, k in enumerate(kept):
        idx[r, : len(k)] = k
    mass = torch.rand(len(lengths), max(lengths) + 1, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((len(lengths), keep + 2), -3.0, device="cuda")
    got = api.mla_kv_compact(
        dev, torch.as_tensor(w.page_table, device="cuda"),
        torch.as_tensor(w.seq_lens, device="cuda"), torch.as_tensor(out_table, device="cuda"),
        torch.as_tensor(idx, device="cuda"),
        torch.as_tensor(np.array([len(k) for k in kept], dtype=np.int32), device="cuda"),
        mass=mass, mass_out=out, status=status)
    assert got is out and int(status.item()) == 0
    want = [oracle.kv_compact(p, w.page_table, out_table, kept) for p in pools]
    for l, x in enumerate(dev):
        bits = x.view(torch.uint8 if fp8 else torch.int16).cpu().numpy()
        assert np.array_equal(bits.view(pools[0].dtype), want[l % len(pools)]), l
    for r, k in enumerate(kept):
        assert torch.equal(out[r, : len(k)], mass[r, torch.as_tensor(k, dtype=torch.long).cuda()])
        assert bool((out[r, len(k):] == -3).all())


def test_bad_indices_and_pages_are_skipped_and_reported():
    w = inputs.custom_workload([100, 2000], 1, 16, seed=1)
    pool = _pool(w, False, 2)
    good = [[3, 50, 99], [0, 1600, 1999]]
    out_table = _fresh(w, [3, 3], 2)

    def run(idx=good, ids=w.page_table, outs=out_table):
        dev = torch.from_numpy(pool.view(np.int16)).cuda().view(torch.bfloat16)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        api.mla_kv_compact([dev], torch.as_tensor(ids, device="cuda"),
                           torch.as_tensor(w.seq_lens, device="cuda"),
                           torch.as_tensor(outs, device="cuda"),
                           torch.tensor(idx, dtype=torch.int32, device="cuda"),
                           torch.tensor([3, 3], dtype=torch.int32, device="cuda"), status=status)
        got = dev.view(torch.int16).cpu().numpy().view(np.uint16)
        return int(status.item()), got

    code, full = run()
    assert code == 0
    for bad in (-1, 100, 2**31 - 1):
        code, got = run([[3, bad, 99], good[1]])
        page = int(out_table[0, 0])
        assert code == 33
        assert np.array_equal(got[page, ROW:2 * ROW], pool[page, ROW:2 * ROW])
        got[page, ROW:2 * ROW] = full[page, ROW:2 * ROW]
        assert np.array_equal(got, full)
    for bad in (-1, w.num_pages + 2, 2**31 - 1):
        ids = np.array(w.page_table)
        ids[1, 1] = bad
        code, got = run(ids=ids)
        page = int(out_table[1, 0])
        assert code == 33 and np.array_equal(got[page, ROW:3 * ROW], pool[page, ROW:3 * ROW])
        outs = np.array(out_table)
        outs[1, 0] = bad
        code, got = run(outs=outs)
        assert code == 33 and np.array_equal(got[page], pool[page])


def test_a_server_step_with_eviction():
    """Append with rotation, decode, accumulate, then select, compact and decode the
    shorter histories, in both cache formats' bf16 form against the oracle: the
    decode after the eviction equals the oracle's attention over the kept rows."""
    R, H, steps, keep = 3, 16, 4, 600
    start = np.array([1534, 700, 2100])
    lens = start + steps
    w = inputs.custom_workload([int(v) for v in lens], 1, H, seed=12, spare_pages=6)
    slab = inputs.make_slab(w, "cuda", poison_nan=False)
    ids = torch.as_tensor(w.page_table, device="cuda")
    table = api.rope_table(64, base=50000.0)
    g = torch.Generator().manual_seed(1)
    mass = torch.zeros(R, int(lens.max()), device="cuda")
    ws = api.allocate_workspace(R, 1, H)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for s in range(steps):
        now = torch.as_tensor((start + s + 1).astype(np.int32), device="cuda")
        rows = [torch.randn(R, n, generator=g).to(torch.bfloat16).cuda() for n in (512, 64)]
        q = torch.randn(R, H, 576, generator=g).to(torch.bfloat16).cuda()
        qr = api.mla_kv_append_rope(*rows, slab, ids, now, 1, table, q_rope=q[..., 512:],
                                    status=status)
        qn = q[..., :512].contiguous()
        out, lse = api.mla_decode(qn, qr, qn, slab, ids, now, workspace=ws)
        api.mla_attention_mass(qn, qr, lse, slab, ids, now, mass, status=status)
    total = mass.double().sum(1).cpu().numpy()
    assert np.all(np.abs(total / (steps * H) - 1.0) <= math.exp(2e-3) - 1.0)

    kept, n = api.mla_evict_select(mass, now, keep, sink=4, recent=64)
    assert n.tolist() == [min(int(v), keep) for v in lens]
    want = oracle.evict_select(mass.cpu().numpy(), lens, keep, 4, 64)
    assert [kept[r, : len(k)].tolist() for r, k in enumerate(want)] == want
    free = [p for p in range(w.num_pages) if p not in set(w.page_table[w.page_table >= 0].tolist())]
    fresh = torch.tensor([[p] for p in free[:R]], dtype=torch.int32, device="cuda")
    carried = api.mla_kv_compact([slab], ids, now, fresh, kept, n, mass=mass, status=status)
    for r, k in enumerate(want):
        assert torch.equal(carried[r, : len(k)], mass[r, torch.tensor(k).cuda()])

    # the next step: the new token's position is not its row
    n1 = n + 1
    rows = [torch.randn(R, d, generator=g).to(torch.bfloat16).cuda() for d in (512, 64)]
    q = torch.randn(R, H, 576, generator=g).to(torch.bfloat16).cuda()
    qr = api.mla_kv_append_rope(*rows, slab, fresh, n1, 1, table, positions=now, status=status,
                                q_rope=q[..., 512:])
    qn, gate = q[..., :512].contiguous(), torch.randn(R, H, 512, generator=g).to(torch.bfloat16)
    out, lse = api.mla_decode(qn, qr, gate.cuda(), slab, fresh, n1)
    assert int(status.item()) == 0
    ref_out, ref_lse = oracle.mla_decode_reference(
        qn.cpu(), qr.cpu(), gate, slab.cpu(), fresh.cpu().numpy(), n1.cpu().numpy(), 1, H, SCALE,
        num_pages=w.num_pages)
    assert_parity(out, lse, ref_out, ref_lse, what="decode after eviction")


def test_front_end_refusals():
    mass = torch.zeros(2, 50, device="cuda")
    lens = torch.full((2,), 50, dtype=torch.int32, device="cuda")
    bad = [
        lambda: api.mla_evict_select(mass, lens, 0),
        lambda: api.mla_evict_select(mass, lens, 10, sink=6, recent=5),
        lambda: api.mla_evict_select(mass, lens, 10, sink=-1),
        lambda: api.mla_evict_select(mass, lens, 1 << 31),
        lambda: api.mla_evict_select(mass[:, ::2], lens, 10),
        lambda: api.mla_evict_select(mass, lens, 10, workspace=torch.zeros(9)),
        lambda: api.mla_evict_select(mass.half(), lens, 10),
        lambda: api.mla_evict_select(mass, lens[:1], 10),
        lambda: api.mla_evict_select(mass, lens, 10,
                                     kept=torch.zeros(2, 9, dtype=torch.int32, device="cuda")),
    ]
    slab = torch.zeros(3, PT * ROW, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    outs = torch.tensor([[2], [2]], dtype=torch.int32, device="cuda")
    kept, n = api.mla_evict_select(mass, lens, 10)

    def compact(slabs=(slab,), outs=outs, **kw):
        return api.mla_kv_compact(list(slabs), ids, lens, outs, kept, n, **kw)
    bad += [
        lambda: compact(()), lambda: compact((slab, slab[:2])),
        lambda: compact((slab, slab.view(torch.uint8))),
        lambda: compact(mass=mass, mass_out=mass), lambda: compact(mass_out=mass),
        lambda: compact(mass=mass, mass_out=torch.zeros(2, 9, device="cuda")),
        lambda: compact(outs=outs.long()),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(RuntimeError):
        compact(outs=ids)
