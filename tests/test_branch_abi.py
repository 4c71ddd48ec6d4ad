"""Host side of the entry points for several continuations of one prompt, and their oracle
(CPU only: every call here is refused, or is host arithmetic, before anything is launched)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from paged_latent_attention_gb300 import _native, api
from paged_latent_attention_gb300.build import build_library

FAKE = 1 << 20            # an aligned address that no call gets to use
PAGE = 1536 * 576


@pytest.fixture(scope="module")
def lib():
    build_library()
    return _native.lib()


def _refuses(call, base, cases):
    for kw in cases:
        assert call(**{**base, **kw}) == 1, kw


def test_fork_and_free_arguments(lib):
    base = dict(table=FAKE, ld=4, cols=3, lens=FAKE, R=2, parents=FAKE, N=2, counts=FAKE, pages=8,
                out=2 * FAKE, out_ld=4, out_cols=3, out_lens=2 * FAKE, st=None)

    def fork(**a):
        return lib.mla_pages_fork(a["table"], a["ld"], a["cols"], a["lens"], a["R"], a["parents"],
                                  a["N"], a["counts"], a["pages"], a["out"], a["out_ld"],
                                  a["out_cols"], a["out_lens"], a["st"], None)
    _refuses(fork, base, [
        dict(table=None), dict(table=FAKE + 2), dict(ld=2), dict(cols=0), dict(lens=None),
        dict(lens=FAKE + 1), dict(R=0), dict(R=1025), dict(parents=None), dict(parents=FAKE + 2),
        dict(N=0), dict(N=1025), dict(counts=None), dict(counts=FAKE + 1), dict(pages=0),
        dict(pages=1 << 31), dict(out=None), dict(out_ld=2), dict(out_cols=0), dict(out_lens=None),
        dict(out=FAKE), dict(out_lens=FAKE), dict(st=FAKE + 1)])

    def free(**a):
        return lib.mla_pages_free(a["table"], a["ld"], a["cols"], a["lens"], a["R"], a["counts"],
                                  a["pages"], a["st"], None)
    _refuses(free, base, [dict(table=None), dict(ld=2), dict(cols=0), dict(lens=None), dict(R=0),
                          dict(R=1025), dict(counts=None), dict(pages=0), dict(st=FAKE + 3)])


def test_reserve_arguments(lib):
    base = dict(layers=2, slabs=[FAKE, FAKE], es=2, pages=8, stride=PAGE, table=FAKE, ld=4, cols=3,
                lens=FAKE, R=2, n=1, each=None, counts=FAKE, work=FAKE, size=1 << 20, st=None)

    def call(**a):
        p = None if a["slabs"] is None else (ctypes.c_void_p * max(len(a["slabs"]), 1))(*a["slabs"])
        return lib.mla_pages_reserve(a["layers"], p, a["es"], a["pages"], a["stride"], a["table"],
                                     a["ld"], a["cols"], a["lens"], a["R"], a["n"], a["each"],
                                     a["counts"], a["work"], a["size"], a["st"], None)
    _refuses(call, base, [
        dict(layers=0), dict(layers=1025), dict(slabs=None), dict(slabs=[FAKE, None]),
        dict(slabs=[FAKE, FAKE + 8]), dict(es=4), dict(pages=0), dict(stride=PAGE - 8),
        dict(stride=PAGE + 4), dict(es=1, stride=PAGE + 8), dict(table=None), dict(ld=2),
        dict(cols=0), dict(lens=None), dict(R=0), dict(R=1025), dict(n=-1), dict(each=FAKE + 2),
        dict(counts=None), dict(work=None), dict(work=FAKE + 16), dict(st=FAKE + 2)])
    size = lib.mla_pages_workspace_size(2)
    assert call(**{**base, "size": size - 1}) == 3
    assert lib.mla_pages_workspace_size(0) == 0 and lib.mla_pages_workspace_size(1025) == 0
    assert size < lib.mla_pages_workspace_size(1024) <= 1024 * 16 + 512


def test_shapes_that_no_workspace_serves(lib):
    """(Sizes need a device; a shape that no kernel takes has none on any.)"""
    for shape in ((0, 1, 64, 1, 0), (1025, 1, 64, 1, 0), (1, 0, 64, 1, 0), (1, 257, 64, 1, 0),
                  (1, 1, 0, 1, 0), (1, 1, 129, 1, 0), (1, 1, 64, 0, 0), (1, 1, 64, 1025, 1)):
        assert lib.mla_shared_workspace_size(*shape) == 0
    assert lib.mla_beam_workspace_size(1, 1, 1) > 0            # (the same on any)
    for shape in ((0, 4, 10), (1, 0, 10), (1, 65, 10), (1, 4, 0), (16384, 4, 10), (1, 64, 1 << 30)):
        assert lib.mla_beam_workspace_size(*shape) == 0


def test_beam_arguments(lib):
    base = dict(x=FAKE, ld=50, dt=0, scores=FAKE, ended=None, end=-1, B=2, K=3, V=50, tok=3 * FAKE,
                par=4 * FAKE, out=2 * FAKE, work=FAKE, size=1 << 30)

    def call(**a):
        return lib.mla_beam_select(a["x"], a["ld"], a["dt"], a["scores"], a["ended"], a["end"],
                                   a["B"], a["K"], a["V"], a["tok"], a["par"], a["out"], a["work"],
                                   a["size"], None)
    _refuses(call, base, [
        dict(x=None), dict(x=FAKE + 1), dict(x=FAKE + 2, dt=2), dict(ld=49), dict(dt=3), dict(dt=-1),
        dict(scores=None), dict(scores=FAKE + 2), dict(ended=FAKE), dict(ended=FAKE, end=50),
        dict(B=0), dict(K=0), dict(K=65), dict(V=0), dict(B=30000), dict(V=1 << 30, ld=1 << 30),
        dict(tok=None), dict(par=FAKE + 1), dict(out=None), dict(out=FAKE), dict(work=None),
        dict(work=FAKE + 128), dict(tok=4 * FAKE), dict(par=3 * FAKE), dict(out=3 * FAKE),
        dict(out=4 * FAKE)])


@pytest.mark.parametrize("fp8", [False, True])
def test_shared_decode_arguments(lib, fp8):
    base = dict(qn=FAKE, qr=FAKE, gate=FAKE, slab=FAKE, pages=8, stride=PAGE, table=FAKE, ld=3,
                cols=2, lens=FAKE, R=2, nq=1, H=64, starts=FAKE, shared=FAKE, G=1, scale=0.1,
                out=FAKE, lse=None, work=FAKE, size=1 << 30, st=None, kv=0.5)

    def call(**a):
        head = (a["qn"], a["qr"], a["gate"], a["slab"], a["pages"], a["stride"])
        tail = (a["table"], a["ld"], a["cols"], a["lens"], a["R"], a["nq"], a["H"], a["starts"],
                a["shared"], a["G"], a["scale"], a["out"], a["lse"], a["work"], a["size"], a["st"],
                None)
        if fp8:
            return lib.mla_decode_shared_fp8(*head, a["kv"], *tail)
        return lib.mla_decode_shared(*head, *tail)
    cases = [dict(qn=None), dict(qn=FAKE + 8), dict(qr=None), dict(qr=FAKE + 8), dict(gate=None),
             dict(gate=FAKE + 4), dict(slab=None), dict(slab=FAKE + 8), dict(pages=0),
             dict(pages=1 << 31), dict(stride=PAGE - 16), dict(stride=PAGE + 4), dict(table=None),
             dict(table=FAKE + 1), dict(cols=0), dict(ld=1), dict(lens=None), dict(R=0),
             dict(R=1025), dict(nq=0), dict(nq=257), dict(H=0), dict(H=129), dict(starts=None),
             dict(starts=FAKE + 2), dict(shared=None), dict(G=0), dict(G=1025), dict(scale=0.0),
             dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(out=None),
             dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(work=None), dict(work=FAKE + 16),
             dict(st=FAKE + 1)]
    if fp8:
        cases += [dict(kv=0.0), dict(kv=-1.0), dict(kv=math.nan), dict(stride=PAGE + 8)]
    _refuses(call, base, cases)


def test_tensors_off_the_device_are_refused():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    x = torch.zeros(2, 4, 512, dtype=torch.bfloat16)
    slab = torch.zeros(1, PAGE, dtype=torch.bfloat16)
    calls = [
        lambda: api.mla_pages_fork(i(2, 3), i(2), i(2), i(4), i(2, 3), i(2)),
        lambda: api.mla_pages_free(i(2, 3), i(2), i(4)),
        lambda: api.mla_pages_reserve([slab], i(2, 3), i(2), 1, i(1)),
        lambda: api.mla_beam_select(torch.zeros(4, 9), torch.zeros(2, 2)),
        lambda: api.mla_decode_shared(x, x[..., :64], x, slab, i(2, 3), i(2), i(2), i(1)),
        lambda: api.mla_decode_shared_fp8(x, x[..., :64], x, slab, i(2, 3), i(2), i(2), i(1),
                                          kv_scale=1.0)]
    for call in calls:
        with pytest.raises(ValueError):
            call()


def test_gradients_are_not_lost_without_a_word():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    x = torch.zeros(2, 4, 512, dtype=torch.bfloat16)
    slab = torch.zeros(1, PAGE, dtype=torch.bfloat16)
    y = x.clone().requires_grad_()
    for q, gate in ((y, x), (x, y)):
        with pytest.raises(ValueError, match="autograd"):
            api.mla_decode_shared(q, x[..., :64], gate, slab, i(2, 3), i(2), i(2), i(1))


# --------------------------------------------------------------------------
# the oracle, by hand
# --------------------------------------------------------------------------

def test_oracle_forks_count_like_assignments():
    table = [[4, 5], [6, 0]]
    out, n, c = oracle.pages_fork(table, [2000, 100], [1, 0, -1], [0, 0, 0, 3, 1, 1, 1],
                                  [[3, 9], [3, 9], [3, 9]], [5, 5, 5])
    assert out.tolist() == [[6, 9], [4, 5], [3, 9]] and n.tolist() == [100, 2000, 0]
    assert c.tolist() == [0, 0, 0, 0, 2, 2, 2]


def test_oracle_reservations_copy_all_but_the_last_holder():
    slab = np.zeros((6, PAGE), np.float32)
    slab[2, : 7 * 576] = np.arange(7 * 576)
    pools, out, c, ok = oracle.pages_reserve([slab], [[2, 8], [2, 8], [2, 8]], [7, 7, 7], [1, 0, 1536],
                                             [1, 0, 3, 0, 0, 1])
    # row 0 copies into page 1; row 1 needs nothing; row 2 copies into 3 and grows into 4
    assert out.tolist() == [[1, 8], [2, 8], [3, 4]] and ok == [True] * 3
    assert c.tolist() == [1, 1, 1, 1, 1, 1]
    assert np.array_equal(pools[0][1, : 7 * 576], slab[2, : 7 * 576])
    assert np.array_equal(pools[0][3, : 7 * 576], slab[2, : 7 * 576])
    _, out, c, ok = oracle.pages_reserve([slab], [[0, 8], [5, 8]], [1536, 1536], [1, 1], [1] * 5 + [0])
    assert out.tolist() == [[0, 5], [5, 8]] and ok == [True, False]


def test_oracle_selection_by_brute_force():
    g = np.random.default_rng(3)
    x = np.round(2 * g.standard_normal((6, 7)))          # many ties
    s = np.array([[0.0, -1.0, -1.0], [-2.0, -2.0, -math.inf]])
    ended = np.array([[False, True, False], [False, False, False]])
    tokens, parents, best = oracle.beam_select(x, s, ended, 4)
    for b in range(2):
        every = []
        for k in range(3):
            row = x[3 * b + k]
            lse = math.log(sum(math.exp(v) for v in row))
            for v in range(7):
                c = s[b, k] + row[v] - lse
                if ended[b, k]:
                    c = s[b, k] if v == 4 else -math.inf
                every.append((-c, 7 * k + v))
        want = sorted((round(c, 9), i) for c, i in every)[:3]
        assert [int(p - 3 * b) * 7 + int(t) for t, p in zip(tokens[b], parents[b])] == \
            [i for _, i in want]
        assert np.allclose(best[b], [-c for c, _ in want])
