"""Refusals of the cache-budget entries that take a page table's columns apart from its
row stride (CPU only: every call here is refused before anything is launched)."""
import ctypes

import pytest

from paged_latent_attention_gb300 import _native
from paged_latent_attention_gb300.build import build_library

FAKE = 1 << 20            # an aligned address that no call gets to use
PAGE = 1536 * 576


@pytest.fixture(scope="module")
def lib():
    build_library()
    return _native.lib()


COLUMNS = [dict(ld=4, cols=0), dict(ld=4, cols=5), dict(ld=4, cols=-1), dict(ld=0, cols=1)]


@pytest.mark.parametrize("kw", COLUMNS)
def test_columns_of_the_page_table(lib, kw):
    table = (FAKE, kw["ld"], kw["cols"], FAKE, 2)
    rope = (1, None, FAKE, 1.0, 0, None, 0, 0, 0, None, None, None)
    assert lib.mla_kv_append_rope_ex(FAKE, FAKE, FAKE, 8, PAGE, *table, *rope) == 1
    assert lib.mla_kv_append_rope_fp8_ex(FAKE, FAKE, FAKE, 8, PAGE, 0.5, *table, *rope) == 1
    pool = (FAKE, FAKE, FAKE, FAKE, 8, PAGE)
    mass = (1, 16, 0.07, 1.0, FAKE, 100, 100)
    assert lib.mla_attention_mass_ex(*pool, *table, *mass, None, None) == 1
    assert lib.mla_attention_mass_fp8_ex(*pool, 0.5, *table, *mass, FAKE, 1 << 20, None, None) == 1
    slabs = ctypes.cast((ctypes.c_void_p * 1)(FAKE), ctypes.c_void_p)
    head = (1, slabs, 2, 8, PAGE)
    tail = (FAKE, 5, FAKE, 2, 5, None, 0, 0, None, 0, None, None)
    good = (4, 4)
    for ids, outs in ((tuple(kw.values()), good), (good, tuple(kw.values()))):
        assert lib.mla_kv_compact_ex(*head, FAKE, *ids, FAKE, 2 * FAKE, *outs, *tail) == 1


def test_status_of_the_selection(lib):
    assert lib.mla_evict_select_ex(FAKE, 100, 100, FAKE, 2, 10, 1, 2, FAKE, 10, FAKE, None, 0,
                                   FAKE + 2, None) == 1
