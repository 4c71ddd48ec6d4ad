"""Outputs that overlap inputs or one another are refused at the C entries too, and what lies
side by side in one buffer is not (CPU only; a call that is not refused for its arguments
is refused for its workspace, or here for want of a device)."""
import ctypes

import pytest
import torch

from paged_latent_attention_gb300 import _native
from paged_latent_attention_gb300.build import build_library

FAKE = 1 << 24
PAGE = 1536 * 576
REFUSED, NO_ROOM = 1, 3


@pytest.fixture(scope="module")
def lib():
    build_library()
    return _native.lib()


def test_beam_outputs(lib):
    def call(tok=FAKE, par=2 * FAKE, out=3 * FAKE, scores=4 * FAKE, ended=None):
        return lib.mla_beam_select(5 * FAKE, 50, 0, scores, ended, 1, 2, 3, 50, tok, par, out,
                                   6 * FAKE, 0, None)
    assert call() == NO_ROOM                         # 24 bytes each
    names = dict(tok=FAKE, par=2 * FAKE, out=3 * FAKE)
    for a in names:
        for b in (*names, "scores"):
            base = names.get(b, 4 * FAKE)
            if a == b:
                continue
            for off in (-20, -4, 0, 4, 20):
                assert call(**{a: base + off}) == REFUSED, (a, b, off)
            for off in (-24, 24):
                assert call(**{a: base + off}) == NO_ROOM, (a, b, off)
        assert call(ended=7 * FAKE, **{a: 7 * FAKE + 4}) == REFUSED
        assert call(ended=7 * FAKE, **{a: 7 * FAKE + 8}) == NO_ROOM


def test_granted_of_a_reservation(lib):
    slabs = (ctypes.c_void_p * 1)(FAKE)

    def call(granted, each=None):
        return lib.mla_pages_reserve_ex(1, slabs, 2, 8, PAGE, 2 * FAKE, 4, 3, 3 * FAKE, 4, 1, each,
                                        granted, 4 * FAKE, 5 * FAKE, 0, None, None)
    assert call(6 * FAKE) == NO_ROOM
    for off in (-12, 0, 4, 12):
        assert call(3 * FAKE + off) == REFUSED
        assert call(7 * FAKE + off, 7 * FAKE) == (NO_ROOM if off == 0 else REFUSED)
    for off in (-16, 16):
        assert call(3 * FAKE + off) == call(7 * FAKE + off, 7 * FAKE) == NO_ROOM
    # the counts (8) and the table (4 rows of 3 columns)
    for off in (-12, 0, 28):
        assert call(4 * FAKE + off) == REFUSED
    for off in (-12, 0, 8, 40, 56):
        assert call(2 * FAKE + off) == REFUSED
    assert call(4 * FAKE + 32) == call(2 * FAKE + 60) == call(2 * FAKE - 16) == NO_ROOM


# (a fork has no workspace to be refused for: where nothing else stops it, its launch fails for
# want of a device)
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on made-up addresses")


@no_gpu
def test_fork_outputs(lib):
    def call(table=FAKE, ld=10, cols=4, lens=2 * FAKE, R=3, out=3 * FAKE, out_ld=10, out_cols=4,
             out_lens=4 * FAKE, N=2):
        return lib.mla_pages_fork(table, ld, cols, lens, R, 5 * FAKE, N, 6 * FAKE, 8, out, out_ld,
                                  out_cols, out_lens, None, None)
    fine = call()
    assert fine not in (0, REFUSED)
    # columns 4 .. 9 of the same grid are free, above and below
    for off in (4, 6, 10 + 5, -10 + 4, -4, -6):
        assert call(out=FAKE + 4 * off) == fine, off
    for off in (0, 1, 3, 7, 9, 10, -1, -3, -7, -10, 20):
        assert call(out=FAKE + 4 * off) == REFUSED, off
    # one row, or strides that are multiples
    assert call(out=FAKE + 16, N=1, out_ld=4) == fine and call(out=FAKE + 28, N=1, out_ld=4) == REFUSED
    assert call(out=FAKE + 16, out_ld=20) == fine and call(out=FAKE + 4, out_ld=20) == REFUSED
    assert call(out=FAKE + 16, out_ld=15) == REFUSED and call(R=1, N=1, out=FAKE + 12) == REFUSED
    for off in (-4, 0, 4, 8):
        assert call(out_lens=2 * FAKE + off) == REFUSED
    assert call(out_lens=2 * FAKE + 12) == fine and call(out_lens=2 * FAKE - 8) == fine
    # lengths inside a table, or between its rows
    for base in (FAKE, 3 * FAKE):
        for off in (-1, 0, 3, 9, 10, 20):
            assert call(out_lens=base + 4 * off) == (fine if base == 3 * FAKE and off == 20 else REFUSED)
        assert call(out_lens=base + 4 * 6) == call(out_lens=base - 8) == fine
    for off in (-8, 0, 12, 8 * 4, 10 * 4):
        assert call(lens=3 * FAKE + off) == REFUSED
    assert call(lens=3 * FAKE + 16) == call(lens=3 * FAKE - 12) == fine


@no_gpu
def test_decode_outputs(lib):
    rows = 2 * 3

    def call(out=FAKE, gate=2 * FAKE, lse=None):
        return lib.mla_decode_shared(3 * FAKE, 4 * FAKE, gate, 5 * FAKE, 8, PAGE, 6 * FAKE, 4, 4,
                                     7 * FAKE, 2, 1, 3, 8 * FAKE, 9 * FAKE, 1, 0.1, out, lse,
                                     10 * FAKE, 0, None, None)
    fine = call()
    assert fine not in (0, REFUSED)
    assert call(out=2 * FAKE) == fine
    for off in (16, -16, 1024 * (rows - 1)):
        assert call(out=2 * FAKE + off) == REFUSED
    assert call(out=2 * FAKE + 1024 * rows) == fine
    for base in (FAKE, 2 * FAKE):
        assert call(lse=base) == call(lse=base + 1024 * rows - 4) == call(lse=base - 4 * rows + 4) == REFUSED
        assert call(lse=base + 1024 * rows) == call(lse=base - 4 * rows) == fine
