"""Plain restatements of the operators for several continuations of one prompt: page
ownership by counts and beam search's selection (in double precision).

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""
from __future__ import annotations

import math

import numpy as np

from .oracle import DC, DR, PAGE_TOKENS

ROW = DC + DR


def pages_fork(table, lens, parents, counts, out_table, out_lens):
    """(out_table, out_lens, counts) after the assignment, page by page."""
    out, n, c = np.array(out_table), np.array(out_lens), np.array(counts)
    for i, p in enumerate(parents):
        for k in range(-(-int(n[i]) // PAGE_TOKENS)):
            c[out[i, k]] -= 1
        n[i] = lens[p] if p >= 0 else 0
        for k in range(-(-int(n[i]) // PAGE_TOKENS)):
            out[i, k] = table[p][k]
            c[out[i, k]] += 1
    return out, n, c


def pages_reserve(slabs, table, lens, n_new, counts):
    """(slabs, table, counts, rows served) after making room for n_new[r] tokens behind
    each history, row by row."""
    out, c, pools = np.array(table), np.array(counts), [np.array(s) for s in slabs]
    free = [p for p in range(len(c)) if c[p] == 0]
    served = []
    for r, (L, new) in enumerate(zip(lens, n_new)):
        L, new = int(L), int(new)
        have, want = -(-L // PAGE_TOKENS), -(-(L + new) // PAGE_TOKENS)
        if new > 0 and L % PAGE_TOKENS != 0 and c[out[r, have - 1]] < 1:
            served.append(False)            # a page that no one is counted to hold
            continue
        shared = new > 0 and L % PAGE_TOKENS != 0 and c[out[r, have - 1]] > 1
        need = (want - have + (1 if shared else 0)) if new > 0 else 0
        if need > len(free):
            served.append(False)
            free = []                       # later rows that need pages get none either
            continue
        served.append(True)
        if shared:
            old, page = out[r, have - 1], free.pop(0)
            c[old] -= 1
            c[page] = 1
            out[r, have - 1] = page
            width = L % PAGE_TOKENS * ROW
            for s in pools:
                s[page, :width] = s[old, :width]
        for k in range(have, have + need - (1 if shared else 0)):
            out[r, k] = free.pop(0)
            c[out[r, k]] = 1
    return pools, out, c, served


def beam_select(logits, scores, ended=None, end_token=-1):
    """(tokens, parents, scores) of the best candidates: logits [B*K, V], scores [B, K]."""
    x = np.asarray(logits, dtype=np.float64)
    B, K = np.shape(scores)
    V = x.shape[1]
    tokens, parents = np.zeros((B, K), np.int64), np.zeros((B, K), np.int64)
    best = np.zeros((B, K))
    for b in range(B):
        cand = np.full((K, V), -math.inf)
        for k in range(K):
            s, row = float(scores[b][k]), x[b * K + k]
            if ended is not None and ended[b][k]:
                if math.isfinite(s):
                    cand[k, end_token] = s
                continue
            with np.errstate(all="ignore"):
                high = np.max(row)
                shift = s - (high + np.log(np.sum(np.exp(row - high))))
            if math.isfinite(shift):
                cand[k] = row + shift
        flat = cand.reshape(-1)
        pick = np.lexsort((np.arange(flat.size), -flat))[:K]
        tokens[b], parents[b], best[b] = pick % V, b * K + pick // V, flat[pick]
    return tokens, parents, best
