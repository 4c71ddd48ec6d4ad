"""The gate of the decode with shared prefixes over all of its range.

The sigmoid: the exponent's rounding, 2^-18 for gates down to -92.8, gives less than
2^-17 of the value; half a step of bf16 is 2^-8 of it, or 2^-134 where that is more."""
import math

import pytest
import torch

from branch_helpers import KVS, LAT, PT, ROW
from paged_latent_attention_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("R,H", [(2, 3), (40, 64)])
def test_gates_of_any_size(R, H, fp8):
    """All tokens are the same, so the output is the gate's sigmoid times their latent."""
    c = KVS * 64.0 if fp8 else 1.0
    slab = torch.full((1, PT * ROW), 64.0 if fp8 else 1.0, device="cuda")
    slab = slab.to(torch.float8_e4m3fn) if fp8 else slab.bfloat16()
    gate = torch.linspace(-104.0, 104.0, R * H * LAT, device="cuda").view(R, H, LAT)
    gate = gate.bfloat16()
    gate[0, 0, :2], gate[-1, -1, -1] = torch.tensor([-math.inf, math.inf]), math.nan
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    args = (torch.zeros(R, H, LAT, dtype=torch.bfloat16, device="cuda"),
            torch.zeros(R, H, 64, dtype=torch.bfloat16, device="cuda"), gate, slab, i(*[[0]] * R),
            i(*[5] * R), i(0, R), i(5))
    out = api.mla_decode_shared_fp8(*args, kv_scale=KVS)[0] if fp8 else api.mla_decode_shared(*args)[0]
    assert bool(torch.isnan(out[-1, -1, -1]))
    assert out[0, 0, :2].tolist()[0] == 0.0
    want = c / (1.0 + torch.exp(-gate.double()))
    err = (out.double() - want).abs()
    tol = 2.0 ** -8 * want + 2.0 ** -15 * want + 2.0 ** -134 * (1 + 2.0 ** -8)
    bad = ~(err <= tol)
    bad[-1, -1, -1] = False
    assert not bool(bad.any()), (gate[bad][:8].tolist(), out[bad][:8].tolist(), want[bad][:8].tolist())
