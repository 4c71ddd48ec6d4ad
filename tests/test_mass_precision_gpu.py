"""How far the accumulated weights are from 64 bits, over a whole result (2-norm), for each
number of query rows that takes a form of its own.

Bound: the scores, each a sum of 576 products in fp32, may be off by one unit of 2^-23 of
themselves on the side of all, which moves token t's weight by 2^-23 sum_rows w |s|; what
else the arithmetic does (the log-sum-exp's product, the exponent's sum, ex2 within 2^-22,
the sums) rounds each row's weight apart, and adds up to less than 2^-22 over 64 rows and
more.  A sum that is truncated at each of 36 steps without being corrected is off by 4 to
7 such units.
"""
import math

import pytest
import torch

from paged_latent_attention_gb300 import api, inputs

pytestmark = pytest.mark.gpu

PT, ROW = inputs.PAGE_TOKENS, inputs.ROW_ELEMS


def _data(kind, R, P, T, rows, g):
    k = torch.randn(R, P * PT, ROW, device="cuda", generator=g)
    q = torch.randn(R * rows, ROW, device="cuda", generator=g)
    if kind == "aligned":                     # queries and keys share a direction
        d = 0.4 * torch.randn(ROW, device="cuda", generator=g)
        k, q = k + d, q + d
    if kind == "rope":                        # the scores come from the rope part
        q[:, :512] *= 0.1
        q[:, 512:] *= 3.0
    if kind == "spread":                      # tokens and elements of unlike sizes
        k = k * torch.exp(0.5 * torch.randn(R, P * PT, 1, device="cuda", generator=g))
        q = q * torch.exp(0.5 * torch.randn(ROW, device="cuda", generator=g))
    return k, q.to(torch.bfloat16)


@pytest.mark.parametrize("n_q,H", [(1, 64), (1, 128), (4, 64), (8, 64), (32, 64)])
@pytest.mark.parametrize("kind,fp8", [("normal", False), ("aligned", False), ("rope", False),
                                      ("spread", False), ("normal", True), ("aligned", True)])
def test_weights_are_as_near_as_fp32_sums(kind, fp8, n_q, H):
    R, T = 2, 2500
    g = torch.Generator(device="cuda").manual_seed(n_q * H)
    P = -(-T // PT)
    k, q = _data(kind, R, P, T, n_q * H, g)
    k = k.view(R * P, PT * ROW)
    unit = inputs.KV_SCALE_E4M3 if fp8 else 1.0
    slab = (k / unit).clamp(-448, 448).to(torch.float8_e4m3fn) if fp8 else k.to(torch.bfloat16)
    x = (slab.float().double() * unit).view(R, P * PT, ROW)[:, :T]
    scale = float(torch.tensor(1 / math.sqrt(192.0), dtype=torch.float32))
    q = q.view(R, n_q * H, ROW)
    behind = n_q - 1 - torch.arange(n_q, device="cuda").repeat_interleave(H)
    seen = torch.arange(T, device="cuda")[:, None] < T - behind[None]
    lse, want, moved = [], [], []
    for r in range(R):
        s = torch.where(seen, scale * x[r] @ q[r].double().T, -math.inf)
        lse.append(torch.logsumexp(s, 0).float())
        w = torch.exp(s - lse[-1].double())
        want.append(w.sum(1))
        moved.append((w * torch.where(seen, s.abs(), 0.0)).sum(1))
    want, moved = torch.stack(want), torch.stack(moved)
    args = (q[..., :512].reshape(R * n_q, H, 512).contiguous(),
            q[..., 512:].reshape(R * n_q, H, 64).contiguous(),
            torch.stack(lse).view(R * n_q, H), slab,
            torch.arange(R * P, dtype=torch.int32, device="cuda").view(R, P),
            torch.full((R,), T, dtype=torch.int32, device="cuda"), torch.zeros(R, T, device="cuda"))
    if fp8:
        got = api.mla_attention_mass_fp8(*args, n_q=n_q, scale=scale, kv_scale=unit, decay=0.0)
    else:
        got = api.mla_attention_mass(*args, n_q=n_q, scale=scale, decay=0.0)
    error = float((got.double() - want).norm() / want.norm())
    bound = 2.0 ** -23 * float(moved.norm() / want.norm()) + 2.0 ** -22
    assert error <= bound, (error, bound)
