"""The operators for several continuations of one prompt as a server runs them: a small
beam search over a paged cache, its steps against the same search on explicit histories."""
import math

import numpy as np
import pytest
import torch

import oracle
from branch_helpers import KVS, PT, ROW, SCALE, check
from paged_latent_attention_gb300 import api

pytestmark = pytest.mark.gpu

LAYERS, H, V, PAGES = 2, 16, 50, 40


def _weights(seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(V, ROW, generator=g).bfloat16(), torch.randn(H * 512, V, generator=g)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("K,prompts", [(4, [1530, 3071]), (3, [700])])
def test_beam_search_over_shared_pages(K, prompts, fp8):
    """Every step: select, fork, free, reserve, append, decode with the prompt shared.  A
    beam's history is followed on the host; its rows and outputs must be those of that
    history, and the pool must hold each page for exactly the rows that use it."""
    B, steps = len(prompts), 8
    emb, head = _weights(K)
    g = torch.Generator().manual_seed(7 + K)
    dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
    store = (lambda x: (x.float() / KVS).clamp(-448, 448).to(dtype)) if fp8 else (lambda x: x)
    slabs = [torch.full((PAGES, PT * ROW), 0.0).to(dtype).cuda() for _ in range(LAYERS)]
    counts = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
    cols = 5
    table = torch.zeros(B, cols, dtype=torch.int32, device="cuda")
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # the prompts' pages come from the pool like all others
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    api.mla_pages_reserve(slabs, table, zero, lens, counts, status=status)
    rows = [[torch.randn(n, ROW, generator=g).bfloat16() for n in prompts] for _ in range(LAYERS)]
    for l in range(LAYERS):
        for b, n in enumerate(prompts):
            flat = slabs[l].view(torch.uint8).view(PAGES, PT, -1) if fp8 else slabs[l].view(PAGES, PT, ROW)
            t = torch.arange(n, device="cuda")
            x = store(rows[l][b]).cuda()
            flat[table[b].long()[t // PT], t % PT] = x.view(torch.uint8) if fp8 else x
    # a prompt becomes K beams; its own row goes
    beams = torch.zeros(B * K, cols, dtype=torch.int32, device="cuda")
    blens = torch.zeros(B * K, dtype=torch.int32, device="cuda")
    other, olens = beams.clone(), blens.clone()
    parents = torch.arange(B, dtype=torch.int32, device="cuda").repeat_interleave(K)
    api.mla_pages_fork(table, lens, parents, counts, beams, blens, status=status)
    api.mla_pages_free(table, lens, counts, status=status)
    starts = torch.arange(0, B * K + 1, K, dtype=torch.int32, device="cuda")
    shared = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    scores = torch.full((B, K), -math.inf, device="cuda")
    scores[:, 0] = 0.0
    logits = torch.randn(B, V, generator=g).cuda().repeat_interleave(K, 0)
    tokens_of = [[] for _ in range(B * K)]                    # of each beam, on the host
    score_of = scores.double().cpu().numpy()
    emb_d, head_d = emb.cuda(), head.cuda()
    for step in range(steps):
        tokens, parents, scores = api.mla_beam_select(logits, scores)
        want = oracle.beam_select(logits.double().cpu().numpy(), score_of)
        assert np.array_equal(tokens.cpu().numpy(), want[0])
        assert np.array_equal(parents.cpu().numpy(), want[1])
        assert np.allclose(scores.double().cpu().numpy(), want[2], rtol=0, atol=2.0 ** -20 * 40)
        score_of = scores.double().cpu().numpy()
        flat = parents.view(-1)
        tokens_of = [tokens_of[p] + [t] for p, t in zip(flat.tolist(), tokens.view(-1).tolist())]
        api.mla_pages_fork(beams, blens, flat, counts, other, olens, status=status)
        api.mla_pages_free(beams, blens, counts, status=status)
        beams, blens, other, olens = other, olens, beams, blens
        api.mla_pages_reserve(slabs, beams, blens, 1, counts, status=status)
        blens += 1
        x = emb_d[tokens.view(-1).long()]
        for l in range(LAYERS):
            new = (x * (l + 1)).contiguous()
            args = (new[:, :512].contiguous(), new[:, 512:].contiguous(), slabs[l], beams, blens, 1)
            if fp8:
                api.mla_kv_append_fp8(*args, kv_scale=KVS, status=status)
            else:
                api.mla_kv_append(*args, status=status)
        for l in range(LAYERS):
            # the pool's rows are the beam's history
            for i, ts in enumerate(tokens_of):
                b = i // K
                hist = torch.cat([rows[l][b], emb[torch.tensor(ts)] * (l + 1)])
                t = torch.arange(len(hist), device="cuda")
                pool = slabs[l].view(torch.uint8).view(PAGES, PT, -1) if fp8 else \
                    slabs[l].view(PAGES, PT, ROW)
                got = pool[beams[i].long()[t // PT], t % PT].cpu()
                ref = store(hist)
                assert torch.equal(got, ref.view(torch.uint8) if fp8 else ref)
            q = x.repeat(1, H).view(-1, H, ROW) * torch.linspace(0.5, 1.5, H, device="cuda")[None, :, None]
            q = q.bfloat16()
            batch = dict(qn=q[..., :512].contiguous(), qr=q[..., 512:].contiguous(),
                         gate=q[..., :512].flip(-1).contiguous(), slab=slabs[l], table=beams,
                         lens=blens, starts=starts, shared=shared, n_q=1, H=H, fp8=fp8,
                         kv_scale=KVS if fp8 else 1.0, pad=0)
            args = [batch[k] for k in ("qn", "qr", "gate", "slab", "table", "lens", "starts", "shared")]
            out, lse = api.mla_decode_shared_fp8(*args, kv_scale=KVS, status=status) if fp8 else \
                api.mla_decode_shared(*args, status=status)
            check(batch, out, lse)
        logits = out.float().view(B * K, -1) @ head_d / 20.0
        # each page is counted once for every row that holds it
        held = np.zeros(PAGES, np.int64)
        for r, n in zip(beams.cpu().numpy(), blens.tolist()):
            for p in r[: -(-n // PT)]:
                held[p] += 1
        assert np.array_equal(counts.cpu().numpy(), held)
        # and the page that a beam writes to is its own
        last = beams.gather(1, ((blens.long() - 1) // PT)[:, None])[:, 0]
        assert bool((counts[last.long()] == 1).all())
    assert int(status.item()) == 0
    api.mla_pages_free(beams, blens, counts, status=status)
    assert int(status.item()) == 0 and not counts.any()
