"""Weights of the decode with shared prefixes over many orders of magnitude: a token that
takes much of a row's weight before a long history of small ones.

Bound.  Scores as in branch_helpers.bounds: off by d, so weights within e^{2d} - 1.  bf16 weights: each
within 2^-8 of itself.  E4M3: a weight p, scaled so that the largest of its 128 tokens is m with
2^-2 <= m <= 2^8, goes in as E4M3(p) and the rest as E5M2:
  p >= 2^-6       E4M3 leaves at most 2^-4 of p's power of two, of which E5M2 (3 bits) leaves
                  2^-3 of that part's own: at most 2^-8 of p
  2^-10 .. 2^-6   E4M3 (steps of 2^-9) leaves at most 2^-10, E5M2 of that at most 2^-14
  below           E5M2 alone: 2^-3 of p, or half of its smallest step, 2^-17
so |error| <= max(2^-8 p, min(max(2^-3 p, 2^-15 m), 2^-12 m)), with 2^-14 <= 2^-12 m and
2^-17 <= 2^-15 m.  The output is rounded to bf16, 2^-8 of itself, and the products lose 2^-23 of a
sum for each 16 tokens."""
import math

import pytest
import torch

from branch_helpers import KVS, LAT, PT, ROW, SCALE, make_batch, reference
from paged_latent_attention_gb300 import api

pytestmark = pytest.mark.gpu


def _batch(groups, n_q, H, fp8, seed, sinks, spread, height):
    """Rows whose latents have the mean 1 and whose scores are N(0, spread) or so, but for
    the tokens `sinks` of every history, some `height` above, with latents of 0.125."""
    b = make_batch(groups, n_q, H, fp8, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = b["slab"].shape[0]
    rows = torch.zeros(pages, PT, ROW, device="cuda")
    rows[..., :LAT] = 1.0 + 0.5 * torch.randn(pages, PT, LAT, generator=g, device="cuda")
    rows[..., LAT:LAT + 8] = torch.randn(pages, PT, 8, generator=g, device="cuda")
    for r, n in enumerate(b["lens"].tolist()):
        for t in sinks:
            if t < n:
                x = rows[int(b["table"][r, t // PT]), t % PT]
                x[:LAT], x[LAT:], x[LAT + 8:LAT + 16] = 0.125, 0.0, 4.0
    # the prefix's last tokens lie in a page of each member
    starts = b["starts"].tolist()
    for first, end, (shared, _) in zip(starts, starts[1:], groups):
        c, n = shared // PT, shared % PT
        for r in range(first + 1, end):
            rows[int(b["table"][r, c]), :n] = rows[int(b["table"][first, c]), :n]
    b["slab"] = (rows.view(pages, -1) / b["kv_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn) \
        if fp8 else rows.view(pages, -1).bfloat16()
    q = torch.zeros_like(b["qr"], dtype=torch.float32)
    q[..., :8] = spread / SCALE / math.sqrt(8.0) * torch.randn(q[..., :8].shape, generator=g,
                                                               device="cuda").sign()
    q[..., 8:16] = height / SCALE / 32.0
    b["qr"], b["qn"] = q.bfloat16(), torch.zeros_like(b["qn"])
    return b


def _tolerance(b):
    """(reference, tolerance, the first token's weight for each row)."""
    ref, _, terms = reference(b)
    tol, first = torch.zeros_like(ref), torch.zeros(ref.shape[:2], device="cuda")
    rows = torch.as_strided(b["slab"].view(torch.uint8) if b["fp8"] else b["slab"],
                            (b["slab"].shape[0], PT, ROW), (PT * ROW, ROW, 1))
    n_q = b["n_q"]
    for r, n in enumerate(b["lens"].tolist()):
        t = torch.arange(n, device="cuda")
        x = rows[b["table"][r].long()[t // PT], t % PT]
        x = (x.view(torch.float8_e4m3fn) if b["fp8"] else x).double() * b["kv_scale"]
        for j in range(n_q):
            i, seen = r * n_q + j, n - (n_q - 1 - j)
            s = SCALE * torch.cat([b["qn"][i], b["qr"][i]], -1).double() @ x[:seen].T
            w = torch.softmax(s, 1)
            first[i] = w[:, 0]
            e = 2.0 ** -8 * w
            if b["fp8"]:
                most = torch.nn.functional.pad(w, (0, -seen % 128)).view(w.shape[0], -1, 128).amax(2)
                most = most.repeat_interleave(128, 1)[:, :seen]
                e = torch.maximum(e, torch.minimum(torch.maximum(w / 8, 2.0 ** -15 * most),
                                                   2.0 ** -12 * most))
            gate = torch.sigmoid(b["gate"][i].double())
            tol[i] = gate * (e @ x[:seen, :LAT].abs())
    d = 2.0 ** -17 * terms["S"] + 2.0 ** -20 + terms["D"]
    more = (torch.exp(2 * d) - 1)[..., None] + float(b["lens"].max()) / 16 * 2.0 ** -23
    return ref, (1 + 2.0 ** -7) * tol + more * terms["A"] + 2.0 ** -8 * ref.abs(), first


def _check(b):
    args = [b[k] for k in ("qn", "qr", "gate", "slab", "table", "lens", "starts", "shared")]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if b["fp8"]:
        out, _ = api.mla_decode_shared_fp8(*args, kv_scale=KVS, n_q=b["n_q"], status=status)
    else:
        out, _ = api.mla_decode_shared(*args, n_q=b["n_q"], status=status)
    ref, tol, first = _tolerance(b)
    assert int(status.item()) == 0
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    return first


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("groups,n_q,H", [
    ([(13_700, [13_800, 13_900, 14_000, 14_100])], 1, 64), ([(0, [13_800]), (0, [11_001])], 4, 64),
    ([(66_000, [66_100, 66_200])], 1, 16),
    ([(12_800, [12_830 + 7 * i for i in range(48)])], 1, 64)])         # segments of 40 tiles
@pytest.mark.parametrize("share", [0.12, 0.4, 0.62, 0.8])
def test_a_first_token_that_takes_much_of_the_weight(groups, n_q, H, share, fp8):
    n = groups[0][1][0]
    height = math.log(n) + 0.5 + math.log(share / (1 - share))
    first = _check(_batch(groups, n_q, H, fp8, 1, [0], 1.0, height))
    assert bool(((first > share / 2) & (first < (1 + share) / 2)).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("octaves", [6.3, 8.6, 10.6, 12.3, 13.4, 14.6, 20.0, 60.0])
def test_equal_small_weights_behind_a_large_one(octaves, fp8):
    """(Equal weights are all rounded the same way.)"""
    _check(_batch([(0, [9000 + 50 * i]) for i in range(24)], 2, 64, fp8, 2, [0], 0.0, octaves * math.log(2.0)))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("octaves", [9.4, 13.4, 50.0])
def test_large_weights_here_and_there(octaves, fp8):
    """The scale of the weights goes down and up along the history, tile by tile and within."""
    sinks = [0, 700, 701, 2999, 3100, 5000, 5128, 5256, 5384, 9000]
    _check(_batch([(9500, [9700 + i for i in range(32)])], 2, 32, fp8, 3, sinks, 1.0, octaves * math.log(2.0)))
