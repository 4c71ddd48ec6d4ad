"""Which pairs of views count as overlapping (CPU tensors; the check reads addresses,
shapes and strides only), against the elements that they address."""
import itertools

import pytest
import torch

from paged_latent_attention_gb300 import api


def _elements(t):
    at = torch.zeros(t.shape, dtype=torch.long)
    for d, (n, s) in enumerate(zip(t.shape, t.stride())):
        at += (torch.arange(n) * s).view([-1 if e == d else 1 for e in range(t.dim())])
    return set((at + t.storage_offset()).reshape(-1).tolist())


def _refused(a, b):
    try:
        api._check_apart(a, b, "overlap")
    except ValueError:
        return True
    return False


def _views():
    base = torch.zeros(6 * 4 * 24)
    heads = base.view(6, 4, 24)
    yield from (heads[..., i:i + 8] for i in (0, 4, 8, 16))
    yield from (heads[i:i + 3, :, 8:16] for i in (0, 2, 3))
    yield heads[:, :2, :8]
    yield heads[:, 2:, :8]
    yield heads[:1, :, 16:]
    yield heads[..., :8].transpose(0, 1)
    yield heads[:, :1, :8].expand(6, 4, 8)
    rows = base.view(6, 96)
    yield from (rows[:, i:j] for i, j in ((0, 40), (40, 96), (39, 50), (0, 1), (95, 96)))
    yield base[:100]
    yield base[100:]
    yield base.view(36, 16)


def test_views_that_share_elements_are_refused():
    views = list(_views())
    for a, b in itertools.product(views, views):
        if _elements(a) & _elements(b):
            assert _refused(a, b), (a.shape, a.stride(), b.shape, b.stride())


def test_columns_of_one_buffer_are_apart():
    """Parts of the same heads or rows side by side share nothing: rotated parts of wider
    heads, weights and carried weights in one buffer."""
    heads = torch.zeros(6, 4, 24)
    rows = torch.zeros(6, 96)
    for a, b in ((heads[..., :8], heads[..., 8:16]), (heads[..., 16:], heads[..., :8]),
                 (heads[..., :8], heads[1:5, :, 16:]), (rows[:, :40], rows[:, 40:]),
                 (rows[:, 50:], rows[:, 3:50]), (rows[:3], rows[3:])):
        assert not _elements(a) & _elements(b)
        assert not _refused(a, b) and not _refused(b, a)
    with pytest.raises(ValueError):
        api._check_apart(rows[:, :40], rows[:, 39:], "overlap")
