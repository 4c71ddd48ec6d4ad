"""Batches with shared prefixes and a 64-bit reference of their decode, with the terms of
its error bound."""
import math

import numpy as np
import torch

from paged_latent_attention_gb300 import inputs

PT, ROW, LAT = 1536, 576, 512
SCALE = 1.0 / math.sqrt(192.0)
KVS = inputs.KV_SCALE_E4M3
E4M3 = torch.float8_e4m3fn


def make_batch(groups, n_q, H, fp8=False, seed=0, pad=0, spare=2, gain=1.0, device="cuda"):
    """groups: [(shared, [length of each member])], in tokens.  Rows of a prefix's last,
    partly shared page are copied into each member's page; every other row is NaN."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=device).manual_seed(seed)
    starts = np.concatenate([[0], np.cumsum([len(m) for _, m in groups])])
    lens = np.array([n for _, m in groups for n in m], np.int64)
    R = len(lens)
    need = -(-lens // PT)
    cols = int(max(need.max(), 1)) + 1
    top = int(need.sum()) + spare
    ids = rng.permutation(top)
    table = np.full((R, cols), -7, np.int64)
    at, r = 0, 0
    slab = torch.full((top, PT * ROW + pad), math.nan, dtype=torch.bfloat16, device=device)
    rows = torch.as_strided(slab, (top, PT, ROW), (PT * ROW + pad, ROW, 1))

    def fill(page, lo, hi):
        rows[page, lo:hi] = torch.randn(hi - lo, ROW, generator=g, device=device).bfloat16()

    for shared, members in groups:
        first = r
        for n in members:
            # the tokens that this row really has in common with the group's first one
            same = min(shared, n, int(lens[first])) if r > first else 0
            for c in range(-(-n // PT)):
                have = min(n - c * PT, PT)
                take = max(0, min(same - c * PT, PT))
                if take == PT:
                    table[r, c] = table[first, c]
                    continue
                table[r, c] = ids[at]
                at += 1
                if take:
                    rows[table[r, c], :take] = rows[table[first, c], :take]
                fill(table[r, c], take, have)
            r += 1
    scale = 1.0
    if fp8:
        scale = KVS
        slab = (slab.float() / KVS).clamp(-448, 448).to(E4M3)
    T = R * n_q
    make = lambda w: torch.randn(T, H, w, generator=g, device=device)
    ints = lambda x: torch.as_tensor(np.asarray(x, np.int32), device=device)
    return dict(qn=(gain * make(LAT)).bfloat16(), qr=(gain * make(64)).bfloat16(),
                gate=make(LAT).bfloat16(), slab=slab, table=ints(table), lens=ints(lens),
                starts=ints(starts), shared=ints([s for s, _ in groups]), n_q=n_q, H=H,
                fp8=fp8, kv_scale=scale, pad=pad)


def reference(b, scale=SCALE, lens=None):
    """(out, lse, terms) in 64 bits: terms A, B (gated), S (the largest sum |scale q x| of a
    row's scores) and D (the two-part query's share of them)."""
    dev = b["slab"].device
    n_q, H = b["n_q"], b["H"]
    lens = (b["lens"] if lens is None else lens).tolist()
    T = len(lens) * n_q
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device=dev)
    out, lse = z(T, H, LAT), torch.full((T, H), -math.inf, dtype=torch.float64, device=dev)
    A, B, S, D = z(T, H, LAT), z(T, H, LAT), z(T, H), z(T, H)
    pages = torch.as_strided(b["slab"], (b["slab"].shape[0], PT, ROW), (PT * ROW + b["pad"], ROW, 1))
    for r, n in enumerate(lens):
        if n <= 0:
            continue
        t = torch.arange(n, device=dev)
        at = b["table"][r].long()[t // PT]
        x = pages.view(torch.uint8 if b["fp8"] else torch.bfloat16)[at, t % PT] if not b["fp8"] \
            else torch.as_strided(b["slab"].view(torch.uint8), pages.shape, pages.stride())[at, t % PT]
        x = (x.view(E4M3) if b["fp8"] else x).double() * b["kv_scale"]
        for j in range(n_q):
            i, seen = r * n_q + j, n - (n_q - 1 - j)
            if seen <= 0:
                continue
            y = x[:seen]
            q = torch.cat([b["qn"][i], b["qr"][i]], -1).double()
            s = scale * q @ y.T
            lse[i] = torch.logsumexp(s, 1)
            w = torch.exp(s - lse[i][:, None])
            gate = torch.sigmoid(b["gate"][i].double())
            c = y[:, :LAT]
            out[i] = gate * (w @ c)
            A[i] = gate * (w @ c.abs())
            B[i] = gate * w.amax(1, keepdim=True) * c.abs().sum(0)
            S[i] = (scale * q.abs() @ y.abs().T).amax(1)
            if b["fp8"]:
                e = torch.ceil(torch.log2(q.abs().amax(1, keepdim=True) / 448.0))
                off = torch.where((q.abs() < 2.0 ** (e - 2)) & (q != 0), 2.0 ** (e - 10), 0.0)
                D[i] = (scale * off @ y.abs().T).amax(1)
    return out, lse, dict(A=A, B=B, S=S, D=D)


def bounds(b, ref, terms):
    """How far out and lse may be.
    Scores: a chain of at most 40 MMAs, each of which may lose a unit of 2^-23 of a partial
    sum that is at most S: off by d <= 40 2^-23 S < 2^-17 S, and two roundings and the
    exponential add 2^-20; E4M3 queries add D.  Weights are then within e^{2d} - 1.
    Probabilities: rounded to bf16, 2^-8 of themselves; or in two E4M3 parts: the first off by at
    most 2^-4 of p, what the second leaves of that by 2^-4 of it, so 2^-8, and both by
    half of the smallest step, 2 2^-10 of numbers whose largest is at least 2^4: 2^-13 of
    the largest weight.
    Products: one truncation of 2^-23 of the sum for each of L / 16 MMAs (E4M3: as many).
    The output's own rounding: 2^-8 of itself."""
    d = 2.0 ** -17 * terms["S"] + 2.0 ** -20 + terms["D"]
    L = float(max(int(b["lens"].max()), 1))
    rel = 2.0 ** -8 * (1 + 2.0 ** -7) + (torch.exp(2 * d) - 1)[..., None] + L / 16 * 2.0 ** -23
    out = 2.0 ** -8 * ref.abs() + rel * terms["A"]
    if b["fp8"]:
        out = out + 2.0 ** -13 * torch.exp(2 * d)[..., None] * terms["B"]
    return out, d


def check(b, out, lse, scale=SCALE, rows=None, lens=None):
    ref, ref_lse, terms = reference(b, scale, lens)
    tol, tol_lse = bounds(b, ref, terms)
    rows = slice(None) if rows is None else rows
    err = (out.double() - ref).abs()[rows]
    assert bool(torch.isfinite(out[rows].float()).all())
    assert bool((err <= tol[rows]).all()), (float(err.max()), float((err / tol[rows]).max()))
    empty = torch.isneginf(ref_lse)
    assert torch.equal(torch.isneginf(lse)[rows], empty[rows])
    off = torch.where(empty, 0.0, (lse.double() - ref_lse).abs())
    lim = tol_lse + 2.0 ** -23 * ref_lse.abs()
    assert bool((off <= torch.where(empty, 1.0, lim))[rows].all()), float((off / lim)[rows].nan_to_num().max())
    assert not bool(out[empty].any())
