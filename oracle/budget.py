"""Plain restatements, in double precision, of the operators that hold a cache to
a budget: rotary positions, the rotating append, accumulated attention weight,
eviction selection and page compaction.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""
from __future__ import annotations

import math

import numpy as np

from .oracle import DC, DR, PAGE_TOKENS, _as_f64

ROW = DC + DR


def rope_frequencies(dim, base=10000.0, scaling="none", factor=1.0, original_len=0.0, low=1.0,
                     high=32.0):
    """Radians per position of each pair."""
    out = []
    for i in range(dim // 2):
        f = base ** (-2.0 * i / dim)
        if scaling == "linear":
            f = f / factor
        elif scaling == "by_parts":
            turns = original_len * f / (2.0 * math.pi)
            g = min(max((turns - low) / (high - low), 0.0), 1.0)
            f = (1.0 - g) * f / factor + g * f
        out.append(f)
    return np.array(out)


def rope_rotate(x, positions, freqs, layout="half", magnitude=1.0, inverse=False):
    """x [T, H, D] turned by positions [T], through complex numbers."""
    x = np.asarray(x, dtype=np.float64)
    angle = np.asarray(positions, dtype=np.float64)[:, None] * freqs[None]
    z = magnitude * np.exp((-1j if inverse else 1j) * angle)[:, None]
    if layout == "half":
        y = (x[..., : x.shape[-1] // 2] + 1j * x[..., x.shape[-1] // 2:]) * z
        return np.concatenate([y.real, y.imag], axis=-1)
    y = (x[..., 0::2] + 1j * x[..., 1::2]) * z
    return np.stack([y.real, y.imag], axis=-1).reshape(x.shape)


def history_rows(slab, table_row, length):
    """The first `length` token rows of one history, as stored: [length, 576]."""
    rows = [np.asarray(slab[int(table_row[c])]).reshape(-1)[: PAGE_TOKENS * ROW]
            .reshape(PAGE_TOKENS, ROW) for c in range(-(-length // PAGE_TOKENS))]
    return np.concatenate(rows)[:length] if rows else np.zeros((0, ROW), slab.dtype)


def attention_mass(q_nope, q_rope, lse, histories, n_q, scale, mass, decay):
    """mass after the step: `histories` is a list of [L_r, 576] float rows."""
    qn, qr = _as_f64(q_nope), _as_f64(q_rope)
    q = np.concatenate([qn, qr], axis=-1)                       # [R*n_q, H, 576]
    out = np.array(mass, dtype=np.float64)
    for r, x in enumerate(histories):
        L = x.shape[0]
        total = np.zeros(L)
        for j in range(n_q):
            seen = max(0, L - (n_q - 1 - j))
            row = r * n_q + j
            if seen == 0:
                continue
            l = np.asarray(lse[row], dtype=np.float64)
            s = scale * x[:seen].astype(np.float64) @ q[row].T  # [seen, H]
            total[:seen] += np.exp(s[:, np.isfinite(l)] - l[np.isfinite(l)][None]).sum(axis=1)
        out[r, :L] = total if decay == 0.0 else decay * out[r, :L] + total
    return out


def evict_select(mass, lens, keep, sink=0, recent=0):
    """Kept indices of each history (a list of ascending lists)."""
    out = []
    for row, L in zip(np.asarray(mass), lens):
        L = max(0, min(int(L), len(row)))
        if L <= keep:
            out.append(list(range(L)))
            continue
        middle = range(sink, L - recent)
        weight = [-math.inf if math.isnan(row[t]) else float(row[t]) for t in middle]
        nan = [math.isnan(row[t]) for t in middle]
        # heaviest first, numbers before NaN, then by index
        order = sorted(range(len(weight)), key=lambda i: (nan[i], -weight[i], i))
        chosen = sorted(sink + i for i in order[: keep - sink - recent])
        out.append(list(range(sink)) + chosen + list(range(L - recent, L)))
    return out


def kv_compact(slab, table, out_table, kept):
    """The pool after the kept rows of each history were copied to its new pages."""
    out = np.array(slab)
    for r, rows in enumerate(kept):
        for i, t in enumerate(rows):
            src = slice(t % PAGE_TOKENS * ROW, (t % PAGE_TOKENS + 1) * ROW)
            dst = slice(i % PAGE_TOKENS * ROW, (i % PAGE_TOKENS + 1) * ROW)
            out[int(out_table[r, i // PAGE_TOKENS]), dst] = \
                slab[int(table[r, t // PAGE_TOKENS]), src]
    return out
