"""Accumulated attention weight on the GPU against the double-precision oracle.

Tolerance of a token's weight, from the arithmetic: a score's 36 MMA steps each
round the fp32 accumulator by at most 2^-22 of the absolute sum S = sum |q_d x_d|,
so the scaled score is off by D = 36 * 2^-22 * scale * max S; the exponent's factor,
product and the log-sum-exp add 2^-23 of a magnitude below 64 each (in all below
2^-15), ex2 2^-22 relative, and the sums of up to 128 terms per chunk, and of the
chunks, 2^-24 per term of the path: below 2^-16 relative.  A weight is therefore
off by at most e^(D + 2^-14) - 1 of itself, their sum likewise, and the final
product and sum with the old mass by 2^-23 of both.  E4M3 pages add the two-part
query's bound to D: sum_d eps_d |x_d| (helpers.fp8_query_error).
"""
import math

import numpy as np
import pytest
import torch

import oracle
from helpers import SCALE, fp8_query_error, gpu_decode, gpu_decode_fp8, to_device
from paged_latent_attention_gb300 import api, inputs

pytestmark = pytest.mark.gpu


def _case(lengths, n_q, H, fp8, seed=0, **kw):
    w = inputs.custom_workload(lengths, n_q, H, seed=seed, **kw)
    qn, qr, gate = inputs.make_queries(w, "cpu")
    slab = (inputs.make_slab_e4m3 if fp8 else inputs.make_slab)(w, "cpu", poison_nan=True)
    scale = inputs.KV_SCALE_E4M3
    hist = []
    for r, L in enumerate(w.seq_lens):
        raw = slab.view(torch.uint8).numpy() if fp8 else slab.view(torch.int16).numpy()
        rows = oracle.history_rows(raw, w.page_table[r], int(L))
        hist.append(oracle.e4m3_decode(rows) * scale if fp8 else
                    torch.from_numpy(rows.copy()).view(torch.bfloat16).double().numpy())
    # log-sum-exps of the visible scores, as a decode returns them (-inf: none)
    lse = np.full((w.num_tokens, H), -np.inf)
    q = np.concatenate([qn.double().numpy(), qr.double().numpy()], axis=-1)
    for r, x in enumerate(hist):
        for j in range(n_q):
            seen = len(x) - (n_q - 1 - j)
            if seen > 0:
                s = SCALE * x[:seen] @ q[r * n_q + j].T
                m = s.max(axis=0)
                lse[r * n_q + j] = m + np.log(np.exp(s - m).sum(axis=0))
    return w, qn, qr, gate, slab, hist, torch.from_numpy(lse.astype(np.float32))


def _device(w, qn, qr, lse, slab):
    return dict(q_nope_absorbed=qn.cuda(), q_rope=qr.cuda(), lse=lse.cuda(), slab=slab.cuda(),
                page_table=torch.as_tensor(w.page_table, device="cuda"),
                seq_lens=torch.as_tensor(w.seq_lens, device="cuda"))


def _run(d, mass, w, fp8, decay=1.0, **kw):
    if fp8:
        return api.mla_attention_mass_fp8(**d, mass=mass, kv_scale=inputs.KV_SCALE_E4M3,
                                          n_q=w.n_q, decay=decay, **kw)
    return api.mla_attention_mass(**d, mass=mass, n_q=w.n_q, decay=decay, **kw)


def _check(got, before, w, qn, qr, lse, hist, fp8, decay):
    ref = oracle.attention_mass(qn, qr, lse.numpy(), hist, w.n_q, SCALE, before, decay)
    old = np.zeros_like(before, dtype=np.float64) if decay == 0 else decay * before
    q = np.abs(np.concatenate([qn.double().numpy(), qr.double().numpy()], axis=-1))
    eps = fp8_query_error(qn, qr).reshape(q.shape) if fp8 else np.zeros_like(q)
    for r, x in enumerate(hist):
        L = len(x)
        if L == 0:
            assert np.array_equal(got[r], before[r])
            continue
        rows = slice(r * w.n_q, (r + 1) * w.n_q)
        per_row = (36 * 2.0 ** -22 * q[rows] + eps[rows]).reshape(-1, q.shape[-1])
        D = SCALE * (np.abs(x) @ per_row.T).max()
        new = ref[r, :L] - old[r, :L]
        tol = (math.exp(D + 2.0 ** -14) - 1) * np.abs(new) + \
            2.0 ** -23 * (np.abs(old[r, :L]) + np.abs(ref[r, :L])) + 1e-37
        err = np.abs(got[r, :L] - ref[r, :L])
        assert np.all(err <= tol), (r, float((err / tol).max()))
        assert np.array_equal(got[r, L:], before[r, L:]), "columns past the history changed"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lengths,n_q,H", [
    ([1], 1, 16), ([1000, 2000], 1, 16), ([127, 128, 129, 0, 1], 1, 64),
    ([1536, 1537, 4608], 1, 48), ([300, 5000], 1, 112), ([700, 2500], 1, 128),
    ([900, 1], 2, 64), ([1, 2, 3, 4, 1537], 4, 64), ([129, 700], 3, 48),
    ([2, 400], 17, 16), ([260, 33], 32, 64), ([3, 300], 256, 16)])
def test_mass_matches_the_oracle(fp8, lengths, n_q, H):
    w, qn, qr, _, slab, hist, lse = _case(lengths, n_q, H, fp8, seed=len(lengths))
    d = _device(w, qn, qr, lse, slab)
    rng = np.random.Generator(np.random.PCG64(1))
    before = rng.random((w.num_reqs, max(lengths) + 5)).astype(np.float32)
    for decay in (1.0, 0.875):
        mass, status = torch.from_numpy(before).cuda(), torch.zeros(1, dtype=torch.int32,
                                                                    device="cuda")
        out = _run(d, mass, w, fp8, decay, status=status)
        assert out is mass and int(status.item()) == 0
        _check(mass.cpu().numpy(), before, w, qn, qr, lse, hist, fp8, decay)
    # decay 0 does not read what was there
    mass = torch.full(before.shape, float("nan"), device="cuda")
    _run(d, mass, w, fp8, 0.0)
    got = mass.cpu().numpy()
    zero = np.zeros_like(before)
    for r, L in enumerate(lengths):
        assert np.all(np.isnan(got[r, L:]))
        got[r, L:] = 0.0
    _check(got, zero, w, qn, qr, lse, hist, fp8, 0.0)


@pytest.mark.parametrize("fp8", [False, True])
def test_many_requests_and_strided_views(fp8):
    """More requests than CTAs, empty ones among them, a page table and a mass that
    are views of wider buffers, padding between pages."""
    rng = np.random.Generator(np.random.PCG64(5))
    lengths = [int(v) for v in rng.integers(0, 260, size=320)]
    w, qn, qr, _, slab, hist, lse = _case(lengths, 1, 16, fp8, seed=2, table_ld=1,
                                          page_stride=inputs.PAGE_TOKENS * inputs.ROW_ELEMS + 64)
    d = _device(w, qn, qr, lse, slab)
    wide = torch.full((320, 7), -1, dtype=torch.int32, device="cuda")
    wide[:, :1] = d["page_table"]
    d["page_table"] = wide[:, :1]
    before = rng.random((320, 300)).astype(np.float32)
    holder = torch.full((320, 500), 3.0, device="cuda")
    mass = holder[:, 50:350]
    mass.copy_(torch.from_numpy(before))
    _run(d, mass, w, fp8)
    _check(mass.cpu().numpy(), before, w, qn, qr, lse, hist, fp8, 1.0)
    assert bool((holder[:, :50] == 3).all()) and bool((holder[:, 350:] == 3).all())


def test_rows_without_weight_and_long_rows_of_pages():
    """A row given lse = -inf adds nothing; a history past its row of mass, its
    table or the pool is reported, and only the tokens inside are updated."""
    w, qn, qr, _, slab, hist, lse = _case([500, 3200], 2, 16, False, seed=3)
    lse[1, 3:9] = -math.inf
    lse[2, :] = -math.inf
    d = _device(w, qn, qr, lse, slab)
    before = np.ones((2, 3300), dtype=np.float32)
    mass = torch.from_numpy(before).cuda()
    _run(d, mass, w, False)
    _check(mass.cpu().numpy(), before, w, qn, qr, lse, hist, False, 1.0)
    full = mass.clone()

    short, status = torch.ones(2, 2000, device="cuda"), torch.zeros(1, dtype=torch.int32,
                                                                    device="cuda")
    _run(d, short, w, False, status=status)
    assert int(status.item()) == 34 and torch.equal(short, full[:, :2000])
    part = torch.ones(2, 3300, device="cuda")
    status.zero_()
    _run({**d, "page_table": d["page_table"][:, :1].contiguous()}, part, w, False, status=status)
    assert int(status.item()) == 33
    assert torch.equal(part[:, :1536], full[:, :1536]) and bool((part[:, 1536:] == 1).all())
    for bad in (-1, w.num_pages, 2**31 - 1):
        ids = d["page_table"].clone()
        ids[1, 0] = bad
        part = torch.ones(2, 3300, device="cuda")
        status.zero_()
        _run({**d, "page_table": ids}, part, w, False, status=status)
        assert int(status.item()) == 33
        same = torch.ones(2, 3300, dtype=torch.bool)
        same[1, :1536] = False
        assert torch.equal(part.cpu()[same], full.cpu()[same])
        assert bool((part[1, :1536] == 1).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_the_weights_of_a_decode_step_sum_to_its_rows(fp8):
    """With the decode's own lse every query row's weights sum to 1, so a request's
    mass sums to n_q * heads: the lse is within 1e-3 (the decode's tolerance; E4M3
    pages add their query bound, below 1e-3 here), the weights within e^(4e-3)."""
    w, qn, qr, gate, slab, hist, _ = _case([5000, 60, 1600], 4, 64, fp8, seed=6)
    dev = to_device(w, qn, qr, gate, slab)
    out, lse = gpu_decode_fp8(w, dev, inputs.KV_SCALE_E4M3) if fp8 else gpu_decode(w, dev)
    mass = torch.zeros(3, 5000, device="cuda")
    _run(_device(w, qn, qr, lse.view(-1, 64).cpu(), slab), mass, w, fp8)
    total = mass.double().sum(1).cpu().numpy()
    assert np.all(np.abs(total / 256.0 - 1.0) <= math.exp(4e-3) - 1.0)


@pytest.mark.parametrize("fp8,n_q", [(False, 1), (False, 4), (True, 1), (True, 4)])
def test_same_bits_streams_and_graphs(fp8, n_q):
    """The same inputs give the same bits: twice, on another stream, in a captured
    and replayed graph; two calls at once on two streams do not disturb each other."""
    w, qn, qr, _, slab, hist, lse = _case([3000, 777, 4100], n_q, 64, fp8, seed=9)
    d = _device(w, qn, qr, lse, slab)
    first = _run(d, torch.zeros(3, 4100, device="cuda"), w, fp8).clone()
    a, b = torch.zeros(3, 4100, device="cuda"), torch.zeros(3, 4100, device="cuda")
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        _run(d, a, w, fp8, 0.0, stream=s1)
        _run(d, b, w, fp8, 0.0, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(a, first) and torch.equal(b, first)
    ws = {"workspace": api.allocate_mass_workspace(3, n_q, 64)} if fp8 else {}
    c = torch.zeros(3, 4100, device="cuda")
    _run(d, c, w, fp8, **ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(d, c, w, fp8, **ws)
    c.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c, first)


def test_layers_accumulate_and_offsets_pass_32_bits():
    """Two layers add into one mass; a page stride of 2^31 bytes and more puts the
    second page beyond 32-bit offsets (an expanded pool of two distant pages)."""
    w, qn, qr, _, slab, hist, lse = _case([2000, 1700], 1, 64, False, seed=4)
    d = _device(w, qn, qr, lse, slab)
    one = _run(d, torch.zeros(2, 2000, device="cuda"), w, False)
    two = _run(d, one.clone(), w, False)
    assert torch.equal(two, one + one)
    far = torch.empty(w.num_pages, 1_200_000_000, dtype=torch.bfloat16, device="cuda")
    far[:, : slab.shape[1]] = d["slab"]
    got = _run({**d, "slab": far}, torch.zeros(2, 2000, device="cuda"), w, False)
    assert torch.equal(got, one)


def test_front_end_refusals():
    w, qn, qr, _, slab, _, lse = _case([100, 50], 1, 16, False)
    d = _device(w, qn, qr, lse, slab)
    mass = torch.zeros(2, 100, device="cuda")
    bad = [
        dict(mass=mass.double()), dict(mass=mass[:1]), dict(mass=mass.t().contiguous().t()),
        dict(mass=mass[:1].expand(2, 100)), dict(lse=d["lse"][:1]), dict(n_q=2),
        dict(n_q=0), dict(seq_lens=d["seq_lens"].long()), dict(page_table=d["page_table"].cpu()),
        dict(slab=d["slab"][:, :-8]), dict(q_rope=d["q_rope"].float()),
        dict(status=torch.zeros(1, device="cuda")),
    ]
    for kw in bad:
        with pytest.raises(ValueError):
            api.mla_attention_mass(**{**d, "mass": mass, **kw})
    for kw in (dict(decay=math.nan), dict(scale=math.inf)):
        with pytest.raises(RuntimeError):
            api.mla_attention_mass(**{**d, "mass": mass, **kw})
    d8 = {**d, "slab": torch.zeros(slab.shape, dtype=torch.uint8, device="cuda")}
    with pytest.raises(ValueError):
        api.mla_attention_mass_fp8(**d8, mass=mass, kv_scale=-1.0)
    with pytest.raises(RuntimeError):
        api.mla_attention_mass_fp8(**d8, mass=mass, kv_scale=1.0,
                                   workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
