"""The rotation under autograd's eyes: refused where a gradient would be lost, the same
values without a graph, and the inverse call as the gradient that autograd finds for the
same map written out in elementary operations."""
import pytest
import torch

from paged_latent_attention_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_inverse_is_autograds_gradient(layout):
    g = torch.Generator().manual_seed(6)
    x, d = (torch.randn(19, 3, 64, generator=g).cuda() for _ in range(2))
    pos = torch.randint(0, 9000, (19,), generator=g, dtype=torch.int32).cuda()
    table = api.rope_table(64, base=50000.0, magnitude=1.5)
    leaf = x.clone().requires_grad_()
    with pytest.raises(ValueError, match="autograd"):
        api.mla_rope(leaf, pos, table, layout=layout)
    with torch.no_grad():
        y = api.mla_rope(leaf, pos, table, layout=layout)
    assert not y.requires_grad and torch.equal(y, api.mla_rope(x, pos, table, layout=layout))

    f = 50000.0 ** (-2.0 * torch.arange(32, dtype=torch.float64, device="cuda") / 64)
    angle = (pos.double()[:, None] * f)[:, None]
    v = leaf.double()
    a, b = v.chunk(2, -1) if layout == "half" else (v[..., 0::2], v[..., 1::2])
    p = 1.5 * (a * angle.cos() - b * angle.sin())
    q = 1.5 * (a * angle.sin() + b * angle.cos())
    z = torch.cat([p, q], -1) if layout == "half" else torch.stack([p, q], -1).flatten(-2)
    (z * d.double()).sum().backward()
    # fp32: below 2^-21 of the magnitude times both elements of the pair, and one rounding
    got = api.mla_rope(d, pos, table, layout=layout, inverse=True)
    tol = 2.0 ** -21 * 1.5 * 2 * d.abs().max() + 2.0 ** -24 * leaf.grad.abs().max()
    assert float((got - leaf.grad).abs().max()) <= float(tol)
