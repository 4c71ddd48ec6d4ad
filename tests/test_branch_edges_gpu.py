"""The largest calls that the operators for continuations of one prompt take, and calls that
share what they may share."""
import math

import numpy as np
import pytest
import torch

import oracle
from branch_helpers import KVS, LAT, PT, ROW, SCALE, bounds, check, make_batch, reference
from paged_latent_attention_gb300 import api

pytestmark = pytest.mark.gpu


def _decode(b, **kw):
    args = [b[k] for k in ("qn", "qr", "gate", "slab", "table", "lens", "starts", "shared")]
    if b["fp8"]:
        return api.mla_decode_shared_fp8(*args, kv_scale=KVS, n_q=b["n_q"], **kw)
    return api.mla_decode_shared(*args, n_q=b["n_q"], **kw)


def _ints(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device="cuda")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("groups,n_q,H", [
    ([(0, [40_000])], 1, 16), ([(60_000, [60_030, 60_200])], 1, 16),
    ([(30_000, [39_000, 41_000, 40_500]), (0, [33_000])], 2, 5)])
def test_rows_of_many_partials(groups, n_q, H, fp8):
    """Few blocks of many tiles: most pairs have a piece of each row."""
    b = make_batch(groups, n_q, H, fp8, seed=3)
    check(b, *_decode(b))


@pytest.mark.parametrize("fp8", [False, True])
def test_a_history_of_all_lengths_there_are(fp8):
    """2^31 - 1 tokens: one page again and again, and 511 tokens of it."""
    b = make_batch([(0, [PT])], 1, 8, fp8, seed=4, spare=0)
    n = 2 ** 31 - 1
    times, rest = divmod(n, PT)
    status = _ints([0])
    long = {**b, "lens": _ints([n]), "table": b["table"][:, :1].repeat(1, times + 1).contiguous()}
    out, lse = _decode(long, status=status)
    assert int(status.item()) == 0
    whole, whole_lse, terms = reference(b)
    gate = torch.sigmoid(b["gate"].double())
    part, part_lse, _ = reference(b, lens=torch.tensor([rest]))
    want_lse = torch.logaddexp(whole_lse + math.log(times), part_lse)
    w = torch.exp(part_lse - want_lse)[..., None]
    want = whole * (1 - w) + part * w
    # A pair adds the terms of its share of the tiles one after another: a rounding of
    # 2^-24 (the weights) or a truncation of 2^-23 for each of 8 MMAs (the products) a tile.
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = -(-n // 128) / (sms // 2) + 2
    tol, tol_lse = bounds(b, want, terms)
    sums = tiles * 2.0 ** -24
    assert bool(((lse.double() - want_lse).abs() <= tol_lse + 1.01 * sums + 2.0 ** -19).all())
    tol = tol + (17.5 * sums) * terms["A"]
    assert bool(((out.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_the_most_requests_with_drafts(fp8):
    """1,024 requests of 8 drafts by 128 heads, of 262,144 tokens and more: more than 2^24
    positions of tiles.  Their pages are four, in different orders."""
    R, n_q, H, pages = 1024, 8, 128, 4
    g = torch.Generator(device="cuda").manual_seed(9)
    make = lambda rows, *s: torch.randn(rows, *s, generator=g, device="cuda", dtype=torch.bfloat16)
    slab = make(pages, PT * ROW)
    if fp8:
        slab = (slab.float() / KVS).clamp(-448, 448).to(torch.float8_e4m3fn)
    lens = 262_144 + torch.arange(R, device="cuda", dtype=torch.int32) % 7 * 40
    table = torch.randint(0, pages, (R, 171), generator=g, device="cuda", dtype=torch.int32)
    b = dict(qn=make(R * n_q, H, LAT), qr=make(R * n_q, H, 64), gate=make(R * n_q, H, LAT), slab=slab,
             table=table, lens=lens, starts=torch.arange(R + 1, device="cuda", dtype=torch.int32),
             shared=torch.zeros(R, device="cuda", dtype=torch.int32), n_q=n_q, H=H, fp8=fp8,
             kv_scale=KVS if fp8 else 1.0, pad=0)
    status = _ints([0])
    out, lse = _decode(b, status=status)
    assert int(status.item()) == 0
    for r, j, h in ((0, 7, 0), (511, 3, 64), (1023, 0, 127), (1022, 7, 1)):
        i = r * n_q + j
        pick = lambda x: x[i:i + 1, h:h + 1].contiguous()
        one = {**b, **{k: pick(b[k]) for k in ("qn", "qr", "gate")}, "n_q": 1, "H": 1,
               "table": table[r:r + 1], "lens": lens[r:r + 1] - (n_q - 1 - j)}
        check(one, pick(out), lse[i:i + 1, h:h + 1])
    seen = lse.view(R, -1)
    assert bool(torch.isfinite(seen).all())


def test_one_workspace_for_calls_one_after_another():
    """Two captured calls and an eager one, on one stream."""
    one = make_batch([(3000, [3100, 3300, 3200])], 1, 64, seed=1)
    two = make_batch([(0, [900]), (700, [800, 1000])], 1, 64, seed=2)
    want = [_decode(one), _decode(two)]
    work = api.allocate_shared_workspace(3, 1, 64, 3)
    graphs, got = [], []
    for b in (one, two):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(_decode(b, workspace=work))
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for out, lse in got:
            out.zero_(), lse.zero_()
        for i in order:
            graphs[i].replay()
        eager = _decode(two, workspace=work)
        assert torch.equal(eager[0], want[1][0])
        for i in order:
            assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1])


def test_empty_requests_behind_a_batch():
    b = make_batch([(900, [1000, 1100]), (0, [0, 0, 0]), (0, [])], 2, 64, seed=5)
    b["lens"][3] = -4
    out, lse = _decode(b)
    check(b, out, lse, lens=b["lens"].clamp(min=0))
    assert not out[4:].any() and bool(torch.isneginf(lse[4:]).all())
    b["lens"].zero_()
    out, lse = _decode(b)
    assert not out.any() and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("K,V,dtype", [
    (1, 2 ** 31 - 1, torch.bfloat16), (64, 33_554_431, torch.bfloat16), (64, 33_554_431, torch.float16),
    (3, 715_827_882, torch.float32)])
def test_the_largest_vocabularies(K, V, dtype):
    x = torch.zeros(K, V, dtype=dtype, device="cuda")
    peaks = sorted({0, 1, V // 2, V // 3, V - 2, V - 1})
    for i, v in enumerate(peaks):
        x[:, v] = 4.0 + 2 * i
    scores = torch.arange(K, device="cuda", dtype=torch.float32)[None] * -16.0
    tokens, parents, best = api.mla_beam_select(x, scores)
    heights = [4.0 + 2 * i for i in range(len(peaks))]
    total = math.log(V - len(peaks) + sum(math.exp(h) for h in heights))
    every = sorted(((float(scores[0, k]) + h - total, -k * V - v, k, v) for k in range(K)
                    for h, v in zip(heights, peaks)), reverse=True)
    # (peaks reach 14 above zero: beams 16 apart come one after the other, zeros between)
    want = []
    for k in range(K):
        mine = [e for e in every if e[2] == k][:K - len(want)]
        want += mine
        v = 0
        while len(want) < K and v < V:              # then this beam's zeros, by token
            if v not in peaks:
                want.append((float(scores[0, k]) - total, 0, k, v))
            v += 1
    assert tokens[0].tolist() == [e[3] for e in want]
    assert parents[0].tolist() == [e[2] for e in want]
    for got, e in zip(best[0].tolist(), want):
        assert abs(got - e[0]) <= 2.0 ** -21 + 2.0 ** -24 * abs(e[0])


@pytest.mark.parametrize("B,K,V", [(65_535, 1, 5), (1023, 64, 70), (20_000, 3, 33)])
def test_the_largest_batches(B, K, V):
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(B * K, V, generator=g, device="cuda")
    scores = torch.randn(B, K, generator=g, device="cuda")
    tokens, parents, best = api.mla_beam_select(x, scores)
    every = (torch.log_softmax(x.double(), 1) + scores.double().view(-1, 1)).view(B, K * V)
    want, at = torch.topk(every, K)
    assert torch.equal(tokens.long(), at % V)
    assert torch.equal(parents.long(), at // V + K * torch.arange(B, device="cuda")[:, None])
    assert bool(((best.double() - want).abs() <= 2.0 ** -21 + 2.0 ** -24 * want.abs()).all())


def test_reservations_of_many_layers_and_rows():
    """More layers than a copy takes, and more pages than a window of the plan."""
    rng = np.random.default_rng(1)
    layers, pages = 70, 7
    table = np.array([[3, 0, 0], [3, 0, 0], [5, 0, 0]], np.int32)
    lens = np.array([700, 701, 1536], np.int32)
    counts = np.array([1, 0, 0, 2, 0, 1, 0], np.int32)
    slabs = [torch.from_numpy(rng.integers(0, 256, (pages, PT * ROW), dtype=np.uint8)).cuda()
             for _ in range(layers)]
    keep = [s.clone() for s in slabs]
    status, t, c = _ints([0]), _ints(table), _ints(counts)
    api.mla_pages_reserve(slabs, t, _ints(lens), 1, c, status=status)
    _, want, left, ok = oracle.pages_reserve([np.zeros((pages, 1), np.uint8)] * 0, table, lens,
                                             [1, 1, 1], counts)
    assert int(status.item()) == 0 and all(ok)
    assert np.array_equal(t.cpu().numpy(), want) and np.array_equal(c.cpu().numpy(), left)
    new = int(want[0, 0])
    for s, k in zip(slabs, keep):
        k[new, :700 * ROW] = k[3, :700 * ROW]
        assert torch.equal(s, k)

    R, pages = 1024, 5000
    lens = rng.integers(0, 2 * PT, R).astype(np.int32)
    table = np.full((R, 6), 77, np.int32)
    counts = (rng.random(pages) < 0.1).astype(np.int32)
    ids = np.flatnonzero(counts == 0)
    rng.shuffle(ids)
    at = 0
    for r in range(R):
        for col in range(-(-int(lens[r]) // PT)):
            table[r, col] = ids[at]
            counts[ids[at]] = 1
            at += 1
    new = rng.integers(0, 3 * PT, R).astype(np.int32)
    slab = torch.empty(pages, PT * ROW, dtype=torch.uint8, device="cuda")
    status, t, c = _ints([0]), _ints(table), _ints(counts)
    api.mla_pages_reserve([slab], t, _ints(lens), _ints(new), c, status=status)
    _, want, left, ok = oracle.pages_reserve([], table, lens, new, counts)
    assert int(status.item()) == (0 if all(ok) else 35)
    assert np.array_equal(t.cpu().numpy(), want) and np.array_equal(c.cpu().numpy(), left)


def test_new_tokens_past_every_table_are_refused():
    slab = torch.empty(2, PT * ROW, dtype=torch.uint8, device="cuda")
    table, counts, status = _ints([[0]]), _ints([1, 0]), _ints([0])
    for n, length in ((2 ** 31 - 1, 5), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1), (1, PT)):
        status.zero_()
        api.mla_pages_reserve([slab], table, _ints([length]), n, counts, status=status)
        assert int(status.item()) == 33 and counts.tolist() == [1, 0] and table.tolist() == [[0]]


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_past_four_gigabytes(fp8):
    """Pages at the end of a pool larger than 2^32 bytes: read, and copied into."""
    pages = 4900 if fp8 else 2450
    b = make_batch([(2000, [2100, 2300]), (0, [1000])], 1, 16, fp8, seed=6, spare=0)
    small, bits = b["slab"].shape[0], torch.uint8 if fp8 else torch.int16
    pool = torch.empty(pages, PT * ROW, dtype=b["slab"].dtype, device="cuda")
    assert pool.numel() * pool.element_size() > 2 ** 32
    pool.view(bits)[pages - small:] = b["slab"].view(bits)
    table = torch.where(b["table"] >= 0, b["table"] + (pages - small), b["table"])
    want = _decode(b)
    got = _decode({**b, "slab": pool, "table": table})
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # page 1 is held twice; the only free page is the last
    counts = torch.ones(pages, dtype=torch.int32, device="cuda")
    counts[1], counts[pages - 1] = 2, 0
    pool.view(bits)[1] = torch.randint(0, 100, (PT * ROW,), dtype=bits, device="cuda")
    rows, status = _ints([[1], [1]]), _ints([0])
    api.mla_pages_reserve([pool], rows, _ints([1400, 1400]), 1, counts, status=status)
    assert int(status.item()) == 0 and rows.tolist() == [[pages - 1], [1]]
    assert torch.equal(pool.view(bits)[pages - 1, :1400 * ROW], pool.view(bits)[1, :1400 * ROW])


def test_calls_refuse_nothing_that_a_view_allows():
    """Tables, counts and lengths that start anywhere in a buffer, rows of logits at any stride."""
    b = make_batch([(1600, [1700, 1650]), (0, [40])], 2, 5, seed=8)
    want = _decode(b)
    shift = {}
    for k in ("lens", "starts", "shared"):
        buf = torch.full((b[k].numel() + 7,), -1, dtype=torch.int32, device="cuda")
        shift[k] = buf[3:3 + b[k].numel()].copy_(b[k])
    wide = torch.full((b["table"].shape[0], b["table"].shape[1] + 5), -1, dtype=torch.int32,
                      device="cuda")
    shift["table"] = wide[:, 1:1 + b["table"].shape[1]].copy_(b["table"])
    got = _decode({**b, **shift})
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    counts = torch.zeros(9, dtype=torch.int32, device="cuda")[1:]        # not 16-byte aligned
    slab = torch.zeros(8, PT * ROW, dtype=torch.uint8, device="cuda")
    table = torch.full((3, 9), -1, dtype=torch.int32, device="cuda")[:, 2:5]
    api.mla_pages_reserve([slab], table, _ints([0, 0, 0]), _ints([PT + 1, 0, 5]), counts)
    assert table.tolist() == [[0, 1, -1], [-1] * 3, [2, -1, -1]]
    assert counts.tolist() == [1, 1, 1, 0, 0, 0, 0, 0]
