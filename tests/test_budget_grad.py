"""Rotations do not lose a gradient without a word (CPU: refused before anything else)."""
import pytest
import torch

from paged_latent_attention_gb300 import api


def _calls(x):
    table = api.RopeTable(torch.zeros(32, dtype=torch.int64), 1.0)
    ids = torch.zeros(1, 1, dtype=torch.int32)
    lens, pos = torch.ones(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    lat, slab = torch.zeros(1, 512), torch.zeros(1, 1536 * 576)
    plain = x.detach().clone()
    yield lambda: api.mla_rope(x, pos, table)
    yield lambda: api.mla_rope(plain, pos, table, out=x)
    for kw in (dict(q_rope=x), dict(q_rope=plain, q_out=x)):
        yield lambda kw=kw: api.mla_kv_append_rope(lat, lat[:, :64], slab, ids, lens, 1, table, **kw)
        yield lambda kw=kw: api.mla_kv_append_rope_fp8(lat, lat[:, :64], slab, ids, lens, 1, table,
                                                       kv_scale=1.0, **kw)


def test_tensors_that_require_grad_are_refused():
    x = torch.zeros(1, 2, 64, requires_grad=True)
    for call in _calls(x):
        with pytest.raises(ValueError, match="autograd"):
            call()
        # without a graph to record, the call goes on to the other checks
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call()
    for call in _calls(x.detach()):
        with pytest.raises(ValueError, match="CUDA"):
            call()
