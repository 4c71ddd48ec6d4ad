"""Which device the eviction's workspace size is asked of (host logic, with stand-ins for
the devices and the library)."""
import contextlib

import pytest
import torch

from paged_latent_attention_gb300 import _native, api


@pytest.fixture
def current(monkeypatch):
    at = [0]

    @contextlib.contextmanager
    def device(d):
        before, at[0] = at[0], d
        yield
        at[0] = before

    class Library:
        @staticmethod
        def mla_evict_workspace_size(num_reqs, tokens):
            return 1000 * (at[0] + 1)

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: at[0])
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: at[0], raising=False)
    monkeypatch.setattr(_native, "lib", Library)
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: (n, str(device)))
    return at


def test_the_size_is_that_of_the_calls_device(current):
    """SM counts and cluster limits differ between devices, so the size of one device may
    be too small, or none, on another."""
    assert api.allocate_evict_workspace(2, 500_000) == (1000, "cuda")
    assert api.allocate_evict_workspace(2, 500_000, device="cuda:2") == (3000, "cuda:2")
    assert api._evict_workspace_size(1, 2, 500_000) == 2000
    assert current == [0]
