"""Refusals of mla_pages_reserve's granted output (CPU only)."""
import ctypes

import pytest
import torch

from paged_latent_attention_gb300 import _native, api
from paged_latent_attention_gb300.build import build_library

FAKE = 1 << 20
PAGE = 1536 * 576


def test_granted_arguments():
    build_library()
    lib = _native.lib()
    slabs = (ctypes.c_void_p * 1)(FAKE)

    def call(granted, lens=FAKE):
        return lib.mla_pages_reserve_ex(1, slabs, 2, 8, PAGE, FAKE, 4, 3, lens, 2, 1, None, granted,
                                        FAKE, FAKE, 1 << 20, None, None)
    assert call(2 * FAKE + 2) == 1 and call(FAKE) == 1


def test_granted_off_the_device_is_refused():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    slab = torch.zeros(1, PAGE, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.mla_pages_reserve([slab], i(2, 3), i(2), 1, i(1), granted=i(2))
