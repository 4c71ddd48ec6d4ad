"""The decode with shared prefixes against 64-bit arithmetic, within a bound derived from
the kernel's roundings (branch_helpers.bounds)."""
import math

import numpy as np
import pytest
import torch

from branch_helpers import KVS, PT, ROW, SCALE, check, make_batch, reference
from paged_latent_attention_gb300 import api

pytestmark = pytest.mark.gpu


def _run(b, **kw):
    args = [b[k] for k in ("qn", "qr", "gate", "slab", "table", "lens", "starts", "shared")]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = kw.pop("want_status", 0)
    if b["fp8"]:
        out, lse = api.mla_decode_shared_fp8(*args, kv_scale=b["kv_scale"], n_q=b["n_q"],
                                             status=status, **kw)
    else:
        out, lse = api.mla_decode_shared(*args, n_q=b["n_q"], status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == want
    return out, lse


GROUPS = {
    "one token": [(0, [1])],
    "one tile": [(128, [129, 128])],
    "pair": [(1500, [1501, 1590])],
    "edges": [(1536, [1537, 1536, 1663]), (127, [200, 128, 127]), (4096, [4097, 4224, 5000])],
    "alone": [(0, [300]), (0, [1]), (5000, [2000]), (0, [1537])],
    "ragged": [(3000, [3001, 4700, 3129]), (0, [77]), (10, [20, 30]), (2999, [3700] * 5)],
    "shared past a member": [(9000, [3000, 2500, 900]), (1000, [1000, 1000])],
    "empty rows": [(0, [0]), (700, [700, 0, 900]), (0, [0, 0]), (500, [501, 502])],
    "empty groups": [(100, []), (2000, [2100, 2200, 2300]), (7, []), (7, [])],
    "many": [(400, [400 + 3 * i for i in range(1, 40)])],
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n_q,H", [(1, 64), (1, 16), (4, 64), (3, 5), (1, 1), (2, 128), (17, 48)])
@pytest.mark.parametrize("name", list(GROUPS))
def test_matches_64_bit_arithmetic(name, n_q, H, fp8):
    b = make_batch(GROUPS[name], n_q, H, fp8, seed=len(name) + H)
    check(b, *_run(b))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("groups,n_q,H", [
    ([(20_011, [20_100 + 211 * i for i in range(8)])], 1, 64),
    ([(9000, [9100 + 37 * i for i in range(12)]), (0, [70_000]), (4000, [4800, 4900])], 4, 64),
    ([(30_000, [30_010, 30_500, 31_000])], 1, 128)])
def test_long_prefixes(groups, n_q, H, fp8):
    b = make_batch(groups, n_q, H, fp8, seed=n_q)
    check(b, *_run(b))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gain", [0.01, 20.0])
def test_small_and_large_scores(gain, fp8):
    """Large scores move the running maximum tile after tile."""
    b = make_batch([(2500, [2600, 3100]), (0, [1800])], 2, 64, fp8, seed=9, gain=gain)
    check(b, *_run(b))


@pytest.mark.parametrize("fp8", [False, True])
def test_scores_that_grow_along_the_history(fp8):
    b = make_batch([(4000, [4100, 4500, 6000])], 1, 16, fp8, seed=4)
    q = torch.cat([b["qn"], b["qr"]], -1).float()[0, 0]
    pages = b["slab"].float() * b["kv_scale"]
    rows = torch.as_strided(pages, (pages.shape[0], PT, ROW), (PT * ROW, ROW, 1))
    for r, n in enumerate(b["lens"].tolist()):
        t = torch.arange(n, device="cuda")
        at = b["table"][r].long()[t // PT]
        rows[at, t % PT] += (t[:, None] / 6000.0) * q[None] * 0.3
    b["slab"] = (pages / KVS).clamp(-448, 448).to(b["slab"].dtype) if fp8 else pages.bfloat16()
    check(b, *_run(b))


def test_agrees_with_the_plain_decode():
    b = make_batch([(3000, [3100, 4000, 3050]), (0, [900])], 2, 64, seed=3)
    out, lse = _run(b)
    ref, ref_lse = api.mla_decode(b["qn"], b["qr"], b["gate"], b["slab"], b["table"], b["lens"], n_q=2)
    check(b, out, lse)
    # both within the same bound of the exact result
    _, _, terms = reference(b)
    assert bool(((out.float() - ref.float()).abs() <= 2.0 ** -6 * terms["A"] + 1e-6).all())
    assert bool(((lse - ref_lse).abs() <= 1e-3).all())


def test_scale_and_no_lse():
    b = make_batch([(600, [700, 640])], 1, 32, seed=5)
    out, lse = _run(b, scale=0.25)
    check(b, out, lse, scale=0.25)
    again, none = _run(b, scale=0.25, with_lse=False)
    assert none is None and torch.equal(out, again)


@pytest.mark.parametrize("fp8", [False, True])
def test_the_same_bits_whatever_the_workspace_held(fp8):
    b = make_batch(GROUPS["ragged"], 2, 64, fp8, seed=6, pad=64)
    out, lse = _run(b)
    check(b, out, lse)
    work = api.allocate_shared_workspace(b["lens"].numel(), 2, 64, b["shared"].numel(), fp8=fp8)
    for fill in (0, 255, 127):
        work.fill_(fill)
        again = _run(b, workspace=work)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = _run(b, stream=side)
    assert torch.equal(out, other[0]) and torch.equal(lse, other[1])


def test_two_calls_at_once():
    """Different batches on two streams, a workspace each."""
    one = make_batch([(9000, [9100 + i for i in range(10)])], 1, 64, seed=1)
    two = make_batch([(0, [5000 + 13 * i]) for i in range(20)], 4, 64, True, seed=2)
    want = [_run(one), _run(two)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for b, s in zip((one, two), streams):
            args = [b[k] for k in ("qn", "qr", "gate", "slab", "table", "lens", "starts", "shared")]
            got.append(api.mla_decode_shared_fp8(*args, kv_scale=KVS, n_q=b["n_q"], stream=s)
                       if b["fp8"] else api.mla_decode_shared(*args, n_q=b["n_q"], stream=s))
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_graph_replay_with_other_groups_and_lengths(fp8):
    batches = [make_batch(g, 1, 64, fp8, seed=11, spare=s) for g, s in [
        ([(1000, [1100, 1200, 1300]), (0, [900])], 0),
        ([(0, [2500]), (2000, [2100, 2000, 2300])], 0)]]
    n = max(b["slab"].shape[0] for b in batches)
    b = dict(batches[0])
    b["slab"] = torch.zeros(n, PT * ROW, device="cuda").to(batches[0]["slab"].dtype)
    b["table"] = torch.zeros(4, max(x["table"].shape[1] for x in batches), dtype=torch.int32,
                             device="cuda")
    work = api.allocate_shared_workspace(4, 1, 64, 2, fp8=fp8)
    graph = torch.cuda.CUDAGraph()
    args = [b[k] for k in ("qn", "qr", "gate", "slab", "table", "lens", "starts", "shared")]
    kw = dict(n_q=1, workspace=work)
    call = (lambda: api.mla_decode_shared_fp8(*args, kv_scale=KVS, **kw)) if fp8 else \
        (lambda: api.mla_decode_shared(*args, **kw))
    keep = {k: b[k].clone() for k in ("qn", "qr", "gate", "lens", "starts", "shared")}
    with torch.cuda.graph(graph):
        out, lse = call()
    for x in (batches[1], {**batches[0], **keep}, batches[1]):
        for k in ("qn", "qr", "gate", "lens", "starts", "shared"):
            b[k].copy_(x[k])
        b["slab"].view(torch.uint8)[:x["slab"].shape[0]].copy_(x["slab"].view(torch.uint8))
        b["table"][:, :x["table"].shape[1]].copy_(x["table"])
        graph.replay()
        torch.cuda.synchronize()
        check(x, out, lse)


@pytest.mark.parametrize("starts", [[1, 2, 4], [0, 3, 2], [0, 2, 5], [0, 2, 3], [0, -1, 4]])
def test_groups_that_are_no_partition_share_nothing(starts):
    b = make_batch([(900, [1000, 1100]), (300, [400, 500])], 1, 64, seed=8)
    want = _run(b)
    b["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    out, lse = _run(b, want_status=38)
    check(b, out, lse)
    b["starts"] = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    again = _run(b)
    assert torch.equal(want[0], again[0])


def test_lengths_and_pages_out_of_range_are_reported():
    b = make_batch([(500, [600, 700]), (0, [1600, 20])], 1, 64, seed=8)
    b["lens"][1] = 5 * PT                           # its row of the table has three columns
    b["table"][1, 1:] = b["table"][0, 0]
    out, _ = _run(b, want_status=33)
    ok = [0, 2, 3]
    ref = reference(b, lens=torch.tensor([600, 0, 1600, 20]))[0]
    assert bool(((out.double() - ref).abs()[ok] <= 0.02).all())
    b = make_batch([(0, [600]), (0, [1600, 20])], 1, 64, seed=8)
    for page in (-3, b["slab"].shape[0], 1 << 30):
        keep = b["table"].clone()
        b["table"][0, 0] = page
        out, _ = _run(b, want_status=33)
        b["table"].copy_(keep)
        ref = reference(b)[0]
        assert bool(((out.double() - ref).abs()[1:] <= 0.02).all())
    b["lens"][0] = -5
    out, lse = _run(b)
    assert not out[0].any() and bool(torch.isneginf(lse[0]).all())


def test_not_a_number_stays_in_its_request():
    b = make_batch([(700, [800, 900]), (0, [1000]), (300, [333, 444])], 1, 64, seed=2)
    page = int(b["table"][2, 0])
    b["slab"].view(-1, PT, ROW)[page, 999, 3] = math.nan
    out, lse = _run(b)
    assert bool(torch.isnan(out[2]).any()) and bool(torch.isnan(lse[2]).any())
    rest = [0, 1, 3, 4]
    b["slab"].view(-1, PT, ROW)[page, 999, 3] = 0.0
    check(b, out, lse, rows=rest)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n_q,H,lens", [
    (2, 64, [129, 640, 1537, 1]), (4, 16, [2, 131, 1538, 4000]), (3, 5, [1536, 1537, 1664, 258]),
    (130, 8, [129, 400, 1600]), (256, 3, [300, 1792])])
def test_drafts_that_see_no_bad_token_stay_clean(n_q, H, lens, fp8):
    """NaN (and infinities) in the cache rows of the last tokens reach the drafts that see them."""
    b = make_batch([(0, [n]) for n in lens], n_q, H, fp8, seed=n_q)
    slab = b["slab"].view(torch.uint8).view(b["slab"].shape[0], PT, -1)
    first = []                                      # the first bad token of each request
    for r, n in enumerate(lens):
        bad = [n - 1] if n_q == 2 else [n - 1, max(n - n_q // 2, 0)]
        for t in bad:
            page, row = int(b["table"][r, t // PT]), t % PT
            x = slab[page, row]
            if fp8:
                x[7 * t % 500], x[t % 512] = 0x7F, 0xFF
            else:
                v = x.view(torch.bfloat16)
                v[7 * t % 500], v[t % 512], v[511] = math.inf, math.nan, -math.inf
        first.append(min(bad))
    out, lse = _run(b)
    clean = [r * n_q + j for r, n in enumerate(lens) for j in range(n_q) if n - (n_q - 1 - j) <= first[r]]
    check(b, out, lse, rows=clean)
    hit = sorted(set(range(len(lens) * n_q)) - set(clean))
    # A score with NaN or +inf among the visible ones leaves no number; one of -inf (two infinities
    # at the same token, by the signs of q) has no weight.
    want = torch.isfinite(reference(b)[1][hit])
    assert torch.equal(torch.isfinite(lse[hit]), want) and not bool(want.all())
    assert torch.equal(torch.isnan(out[hit]), ~want[..., None].expand(-1, -1, 512))


def test_views_and_outputs():
    b = make_batch([(700, [800, 900]), (0, [2000])], 1, 64, seed=2)
    want = _run(b)
    wide = torch.full((3, 9), -1, dtype=torch.int32, device="cuda")
    wide[:, 4:4 + b["table"].shape[1]] = b["table"]
    out = torch.empty_like(b["qn"])
    got = _run({**b, "table": wide[:, 4:4 + b["table"].shape[1]]}, out=out)
    assert got[0] is out and torch.equal(want[0], out) and torch.equal(want[1], got[1])
    # gated in place
    gate = b["gate"].clone()
    got = _run({**b, "gate": gate}, out=gate)
    assert torch.equal(want[0], gate)


def test_refusals():
    b = make_batch([(50, [60, 70])], 1, 16, seed=2)
    names = ("qn", "qr", "gate", "slab", "table", "lens", "starts", "shared")

    def call(**kw):
        x = {**b, **{k: v for k, v in kw.items() if k in names}}
        more = {k: v for k, v in kw.items() if k not in names}
        return api.mla_decode_shared(*[x[k] for k in names], **more)

    call()
    bad = [dict(qn=b["qn"].float()), dict(qn=b["qn"][:, ::2]), dict(qr=b["qr"][:1]),
           dict(gate=b["gate"].cpu()), dict(slab=b["slab"].float()), dict(slab=b["slab"][:, :1000]),
           dict(table=b["table"].long()), dict(table=b["table"][:1]), dict(lens=b["lens"][:1]),
           dict(starts=b["starts"][:1]), dict(starts=b["starts"].long()),
           dict(shared=b["shared"][:0]), dict(shared=b["shared"].cpu()), dict(n_q=3), dict(n_q=0),
           dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf),
           dict(out=torch.empty(2, 16, 512, device="cuda")), dict(lse=torch.empty(2, 15, device="cuda")),
           dict(workspace=torch.empty(1000, dtype=torch.uint8, device="cuda")),
           dict(status=torch.zeros(1, device="cuda")),
           dict(qn=b["qn"].clone().requires_grad_())]
    for kw in bad:
        with pytest.raises((ValueError, RuntimeError)):
            call(**kw)
    with pytest.raises(ValueError):
        api.mla_decode_shared_fp8(*[b[k] for k in names], kv_scale=1.0)
    with pytest.raises(ValueError):
        api.mla_decode_shared_fp8(*[b[k] for k in names], kv_scale=0.0)
