"""Host side of the cache-budget entry points and their oracle (CPU only: every call
here is refused, or is host arithmetic, before anything is launched)."""
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


def _turns(lib, dim=64, base=1e4, scaling=0, factor=1.0, original=0.0, low=1.0, high=32.0):
    out = np.zeros(max(dim, 2) // 2, dtype=np.uint64)
    rc = lib.mla_rope_turns(dim, base, scaling, factor, original, low, high,
                            out.ctypes.data_as(ctypes.c_void_p))
    return rc, out


@pytest.mark.parametrize("dim", [2, 20, 64, 512])
@pytest.mark.parametrize("scaling,kw", [
    ("none", {}), ("linear", dict(factor=7.5)),
    ("by_parts", dict(factor=32.0, original=4096.0, low=1.0, high=32.0))])
def test_rope_turns_follow_the_formula(lib, dim, scaling, kw):
    """turns = f / (2 pi) 2^64, within the few roundings of a double (2^-50 relative)."""
    rc, got = _turns(lib, dim, 5e4, api.ROPE_SCALINGS[scaling], **kw)
    assert rc == 0
    want = oracle.rope_frequencies(dim, 5e4, scaling, kw.get("factor", 1.0),
                                   kw.get("original", 0.0)) / (2 * math.pi) * 2.0 ** 64
    assert np.all(np.abs(got.astype(np.float64) - want) <= 2.0 ** -50 * want + 1)


def test_by_parts_keeps_fast_pairs_and_divides_slow_ones(lib):
    _, plain = _turns(lib)
    _, parts = _turns(lib, scaling=2, factor=8.0, original=4096.0, low=1.0, high=32.0)
    turns = 4096.0 * plain.astype(np.float64) / 2.0 ** 64
    fast, slow = turns > 32, turns < 1
    assert fast.any() and slow.any()
    assert np.allclose(parts[fast] / plain[fast], 1.0) and np.allclose(parts[slow] / plain[slow], 0.125)
    ratio = parts / plain.astype(np.float64)
    assert np.all(np.diff(ratio) <= 1e-12)


@pytest.mark.parametrize("kw", [
    dict(dim=0), dict(dim=3), dict(dim=514), dict(base=1.0), dict(base=math.nan),
    dict(base=math.inf), dict(scaling=3), dict(scaling=-1), dict(scaling=1, factor=0.5),
    dict(scaling=1, factor=math.nan), dict(scaling=2, factor=2.0, original=0.0),
    dict(scaling=2, factor=2.0, original=4096.0, low=4.0, high=4.0),
    dict(scaling=2, factor=2.0, original=4096.0, low=-1.0),
    dict(scaling=2, factor=2.0, original=4096.0, high=math.inf)])
def test_rope_turns_refusals(lib, kw):
    assert _turns(lib, **kw)[0] == 1


def test_rope_table_refusals():
    for kw in (dict(dim=7), dict(scaling="ramp"), dict(magnitude=math.nan),
               dict(scaling="by_parts", factor=2.0)):
        with pytest.raises(ValueError):
            api.rope_table(device="cpu", **kw)
    table = api.rope_table(32, scaling="by_parts", factor=math.e, original_len=4096, device="cpu")
    assert table.dim == 32 and abs(table.magnitude - 1.1) < 1e-12


@pytest.mark.parametrize("turns,magnitude", [
    (torch.zeros(32), 1.0), (torch.zeros(32, dtype=torch.int32), 1.0),
    (torch.zeros(64, dtype=torch.int64)[::2], 1.0),
    (torch.zeros(4, 8, dtype=torch.int64), 1.0),
    (torch.zeros(32, dtype=torch.int64), math.nan)])
def test_rope_tables_of_other_forms_are_refused(turns, magnitude):
    """The kernels read dim / 2 consecutive 64-bit values."""
    with pytest.raises(ValueError):
        api.RopeTable(turns, magnitude)


def test_rope_arguments(lib):
    base = dict(x=FAKE, ts=64, hs=64, pos=FAKE, turns=FAKE, mag=1.0, T=2, H=1, dim=64, dt=0,
                layout=0, inv=0, out=2 * FAKE, ots=64, ohs=64)

    def call(**kw):
        a = {**base, **kw}
        return lib.mla_rope(a["x"], a["ts"], a["hs"], a["pos"], a["turns"], a["mag"], a["T"],
                            a["H"], a["dim"], a["dt"], a["layout"], a["inv"], a["out"], a["ots"],
                            a["ohs"], None)
    for kw in (dict(x=None), dict(out=None), dict(pos=None), dict(turns=None), dict(x=FAKE + 1),
               dict(out=FAKE + 2, dt=2), dict(pos=FAKE + 2), dict(turns=FAKE + 4), dict(T=-1),
               dict(H=0), dict(H=65536), dict(dim=63), dict(dim=0), dict(dim=514), dict(dt=3),
               dict(dt=-1), dict(layout=2), dict(mag=math.inf), dict(mag=math.nan),
               dict(out=FAKE, ots=128)):
        assert call(**kw) == 1, kw
    assert call(T=0, x=None) == 0


def test_rotating_append_arguments(lib):
    base = dict(lat=FAKE, rope=FAKE, slab=FAKE, pages=8, stride=PAGE, ids=FAKE, ld=1, lens=FAKE,
                R=2, n=1, pos=None, turns=FAKE, mag=1.0, layout=0, q=None, ts=64, hs=64, H=1,
                out=None, st=None)

    def call(fp8=False, scale=0.5, **kw):
        a = {**base, **kw}
        head = (a["lat"], a["rope"], a["slab"], a["pages"], a["stride"])
        tail = (a["ids"], a["ld"], a["lens"], a["R"], a["n"], a["pos"], a["turns"], a["mag"],
                a["layout"], a["q"], a["ts"], a["hs"], a["H"], a["out"], a["st"], None)
        if fp8:
            return lib.mla_kv_append_rope_fp8(*head, scale, *tail)
        return lib.mla_kv_append_rope(*head, *tail)
    for kw in (dict(lat=None), dict(rope=FAKE + 8), dict(slab=None), dict(slab=FAKE + 8),
               dict(pages=0), dict(stride=PAGE - 8), dict(stride=PAGE + 4), dict(ids=None),
               dict(ld=0), dict(lens=FAKE + 2), dict(R=0), dict(n=-1), dict(pos=FAKE + 1),
               dict(turns=None), dict(turns=FAKE + 4), dict(mag=math.nan), dict(layout=7),
               dict(q=FAKE), dict(q=FAKE, out=FAKE), dict(q=FAKE, out=2 * FAKE, H=0),
               dict(q=FAKE + 1, out=2 * FAKE), dict(q=FAKE, out=2 * FAKE + 8), dict(st=FAKE + 2)):
        assert call(**kw) == 1, kw
        assert call(fp8=True, **kw) == 1, kw
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert call(fp8=True, scale=scale) == 1
    assert call(fp8=True, stride=PAGE + 8) == 1
    assert call(n=0, lat=None) == 0


def test_mass_arguments(lib):
    base = dict(qn=FAKE, qr=FAKE, lse=FAKE, slab=FAKE, pages=8, stride=PAGE, ids=FAKE, ld=1,
                lens=FAKE, R=2, n_q=1, H=16, scale=0.07, decay=1.0, mass=FAKE, mld=100, cols=100,
                ws=FAKE, bytes=1 << 20, st=None)

    def call(fp8=False, kv=0.5, **kw):
        a = {**base, **kw}
        head = (a["qn"], a["qr"], a["lse"], a["slab"], a["pages"], a["stride"])
        tail = (a["ids"], a["ld"], a["lens"], a["R"], a["n_q"], a["H"], a["scale"], a["decay"],
                a["mass"], a["mld"], a["cols"])
        if fp8:
            return lib.mla_attention_mass_fp8(*head, kv, *tail, a["ws"], a["bytes"], a["st"], None)
        return lib.mla_attention_mass(*head, *tail, a["st"], None)
    for kw in (dict(qn=None), dict(qn=FAKE + 8), dict(qr=None), dict(lse=None), dict(lse=FAKE + 2),
               dict(slab=None), dict(slab=FAKE + 8), dict(pages=0), dict(pages=1 << 31),
               dict(stride=PAGE - 16), dict(stride=PAGE + 4), dict(ids=None), dict(ld=0),
               dict(lens=None), dict(R=0), dict(R=1025), dict(n_q=0), dict(n_q=257), dict(H=24),
               dict(H=144), dict(scale=math.nan), dict(decay=math.inf), dict(mass=None),
               dict(mass=FAKE + 2), dict(cols=0), dict(mld=99), dict(st=FAKE + 1)):
        assert call(**kw) == 1, kw
        assert call(fp8=True, **kw) == 1, kw
    assert call(fp8=True, kv=0.0) == 1
    assert call(fp8=True, stride=PAGE + 8) == 1
    size = lib.mla_mass_workspace_size_fp8(2, 1, 16)
    assert size >= 32 * (2 * 576 + 4) and lib.mla_mass_workspace_size_fp8(2, 0, 16) == 0


def test_select_arguments(lib):
    base = dict(mass=FAKE, ld=100, cols=100, lens=FAKE, R=2, keep=10, sink=1, recent=2, kept=FAKE,
                kld=10, n=FAKE, ws=None)

    def call(**kw):
        a = {**base, **kw}
        return lib.mla_evict_select(a["mass"], a["ld"], a["cols"], a["lens"], a["R"], a["keep"],
                                    a["sink"], a["recent"], a["kept"], a["kld"], a["n"], a["ws"],
                                    0, None)
    for kw in (dict(mass=None), dict(mass=FAKE + 2), dict(ld=99), dict(cols=0), dict(lens=None),
               dict(R=0), dict(R=1025), dict(keep=0), dict(sink=-1), dict(recent=-1),
               dict(sink=5, recent=6), dict(sink=2**31 - 1, recent=2**31 - 1, keep=2**31 - 1),
               dict(kept=None), dict(kld=9), dict(n=None), dict(n=FAKE + 1), dict(ws=FAKE + 128)):
        assert call(**kw) == 1, kw
    assert lib.mla_evict_workspace_size(0, 100) == 0
    assert lib.mla_evict_workspace_size(1, 0) == 0


def test_compact_arguments(lib):
    def array(*ptrs):
        return ctypes.cast((ctypes.c_void_p * len(ptrs))(*ptrs), ctypes.c_void_p)
    base = dict(layers=2, slabs=array(FAKE, FAKE), size=2, pages=8, stride=PAGE, ids=FAKE, ld=1,
                lens=FAKE, outs=2 * FAKE, old=1, kept=FAKE, kld=5, n=FAKE, R=2, cols=5, mass=None,
                mld=0, mcols=0, mout=None, mold=0, st=None)

    def call(**kw):
        a = {**base, **kw}
        return lib.mla_kv_compact(a["layers"], a["slabs"], a["size"], a["pages"], a["stride"],
                                  a["ids"], a["ld"], a["lens"], a["outs"], a["old"], a["kept"],
                                  a["kld"], a["n"], a["R"], a["cols"], a["mass"], a["mld"],
                                  a["mcols"], a["mout"], a["mold"], a["st"], None)
    mass = dict(mass=FAKE, mld=9, mcols=9, mout=2 * FAKE, mold=5)
    for kw in (dict(layers=0), dict(layers=1025), dict(slabs=None), dict(slabs=array(FAKE, None)),
               dict(slabs=array(FAKE, FAKE + 8)), dict(size=4), dict(pages=0),
               dict(stride=PAGE - 8), dict(stride=PAGE + 4), dict(size=1, stride=PAGE + 8),
               dict(ids=None), dict(ld=0), dict(lens=None), dict(outs=None), dict(outs=FAKE),
               dict(old=0), dict(kept=None), dict(kept=FAKE + 2), dict(kld=4), dict(n=None),
               dict(R=0), dict(R=1025), dict(cols=-1), dict(st=FAKE + 2), dict(mass=FAKE),
               dict(mout=FAKE), {**mass, "mout": FAKE}, {**mass, "mld": 8}, {**mass, "mcols": 0},
               {**mass, "mold": 4}, {**mass, "mass": FAKE + 2}):
        assert call(**kw) == 1, kw
    assert call(cols=0) == 0


# ---- the oracle against independent statements --------------------------------------

@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_oracle_rotation_by_hand(layout):
    rng = np.random.Generator(np.random.PCG64(0))
    x, pos = rng.standard_normal((3, 2, 8)), [0, 5, -77]
    f = oracle.rope_frequencies(8)
    got = oracle.rope_rotate(x, pos, f, layout, 1.5)
    for t, p in enumerate(pos):
        for h in range(2):
            for i in range(4):
                a, b = (i, i + 4) if layout == "half" else (2 * i, 2 * i + 1)
                c, s = math.cos(p * f[i]), math.sin(p * f[i])
                u, v = x[t, h, a], x[t, h, b]
                assert abs(got[t, h, a] - 1.5 * (u * c - v * s)) < 1e-12
                assert abs(got[t, h, b] - 1.5 * (u * s + v * c)) < 1e-12
    back = oracle.rope_rotate(got, pos, f, layout, 1 / 1.5, inverse=True)
    assert np.allclose(back, x, atol=1e-12)


def test_oracle_mass_is_the_softmax_summed_over_rows():
    rng = np.random.Generator(np.random.PCG64(1))
    R, n_q, H, L = 2, 3, 2, [5, 2]
    q = rng.standard_normal((R * n_q, H, 576))
    hist = [rng.standard_normal((n, 576)) for n in L]
    lse, want = np.full((R * n_q, H), -np.inf), np.zeros((R, 6))
    for r in range(R):
        for j in range(n_q):
            seen = L[r] - (n_q - 1 - j)
            if seen <= 0:
                continue
            s = torch.from_numpy(0.05 * hist[r][:seen] @ q[r * n_q + j].T)
            lse[r * n_q + j] = torch.logsumexp(s, 0).numpy()
            want[r, :seen] += torch.softmax(s, 0).sum(1).numpy()
    got = oracle.attention_mass(q[..., :512], q[..., 512:], lse, hist, n_q, 0.05,
                                np.ones((R, 6)), 0.5)
    for r in range(R):
        assert np.allclose(got[r, :L[r]], 0.5 + want[r, :L[r]], atol=1e-12)
        assert np.all(got[r, L[r]:] == 1.0)


def test_oracle_selection_small():
    nan = math.nan
    rows = [[3, 1, 2, 2, 0], [nan, -math.inf, 1, nan, 0], [5, 5, 5, 5, 5]]
    assert oracle.evict_select(rows, [5, 5, 5], 3) == [[0, 2, 3], [1, 2, 4], [0, 1, 2]]
    assert oracle.evict_select(rows, [5, 5, 5], 3, 1, 1) == [[0, 2, 4], [0, 2, 4], [0, 1, 4]]
    assert oracle.evict_select(rows, [2, 0, -1], 3) == [[0, 1], [], []]
    assert oracle.evict_select(rows, [9, 5, 5], 2, 1, 1) == [[0, 4], [0, 4], [0, 4]]
