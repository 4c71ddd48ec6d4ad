"""Page ownership on the GPU: forks, releases and reservations, exact against the oracle."""
import numpy as np
import pytest
import torch

import oracle
from paged_latent_attention_gb300 import api

pytestmark = pytest.mark.gpu

PT, ROW = 1536, 576


def _ints(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device="cuda")


def _held(table, lens, pages):
    """Counts of a table's rows alone."""
    counts = np.zeros(pages, np.int32)
    for r, n in enumerate(lens):
        for c in range(-(-int(n) // PT)):
            counts[table[r, c]] += 1
    return counts


def _world(rows, hi, pages, seed, share=True):
    """Rows of up to hi pages; some take their first pages from an earlier row."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, hi * PT + 1, rows)
    lens[rng.random(rows) < 0.2] = hi * PT
    ids = rng.permutation(pages)
    table = np.full((rows, hi + 2), 12345678, np.int64)
    at = 0
    for r in range(rows):
        n = -(-int(lens[r]) // PT)
        k = 0
        if share and r and rng.random() < 0.6:
            k = min(n, -(-int(lens[r - 1]) // PT))
            table[r, :k] = table[r - 1, :k]
        table[r, k:n] = ids[at:at + n - k]
        at += n - k
    counts = _held(table, lens, pages)
    counts[ids[at:][::3]] = 2                       # held elsewhere
    return table.astype(np.int32), lens.astype(np.int32), counts, rng


@pytest.mark.parametrize("rows,out_rows,hi,pages", [
    (1, 1, 1, 4), (1, 9, 3, 64), (4, 4, 2, 100), (7, 3, 200, 2000), (1024, 1024, 5, 9000),
    (130, 1024, 40, 9000)])
def test_fork_matches_the_oracle(rows, out_rows, hi, pages):
    table, lens, counts, rng = _world(rows, hi, pages, rows + hi)
    parents = rng.integers(-1, rows, out_rows).astype(np.int32)
    out = np.full((out_rows, hi + 3), -9, np.int32)
    n = np.zeros(out_rows, np.int32)
    d = dict(table=_ints(table), lens=_ints(lens), counts=_ints(counts), out=_ints(out), n=_ints(n))
    status = _ints([0])
    for _ in range(3):                              # the second gives up what the first took
        out, n, counts = oracle.pages_fork(table, lens, parents, counts, out, n)
        got = api.mla_pages_fork(d["table"], d["lens"], _ints(parents), d["counts"], d["out"],
                                 d["n"], status=status)
        assert got[0] is d["out"] and got[1] is d["n"]
        assert np.array_equal(d["out"].cpu().numpy(), out)
        assert np.array_equal(d["n"].cpu().numpy(), n)
        assert np.array_equal(d["counts"].cpu().numpy(), counts)
        parents = rng.integers(-1, rows, out_rows).astype(np.int32)
    assert int(status.item()) == 0
    assert np.array_equal(d["table"].cpu().numpy(), table)
    api.mla_pages_free(d["out"], d["n"], d["counts"], status=status)
    api.mla_pages_free(d["table"], d["lens"], d["counts"], status=status)
    assert int(status.item()) == 0 and not d["n"].any() and not d["lens"].any()
    left = counts - _held(out, n, pages) - _held(table, lens, pages)
    assert np.array_equal(d["counts"].cpu().numpy(), left)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows,hi,pages,new,layers", [
    (1, 1, 6, 1, 1), (2, 1, 8, 1, 2), (5, 2, 40, 1536, 1), (12, 3, 70, 5, 3), (30, 2, 90, 4000, 1)])
def test_reserve_matches_the_oracle(rows, hi, pages, new, layers, fp8):
    table, lens, counts, rng = _world(rows, hi, pages, rows + new)
    cols = hi + 2 + -(-new // PT)
    wide = np.full((rows, cols), -3, np.int32)
    wide[:, :table.shape[1]] = table
    # every other row is continued twice: a copy of it holds the same pages
    twin = np.arange(rows)[::2]
    wide, lens = np.concatenate([wide, wide[twin]]), np.concatenate([lens, lens[twin]])
    counts = counts + _held(wide[rows:], lens[rows:], pages)
    g = torch.Generator(device="cuda").manual_seed(rows)
    slabs = [torch.randint(0, 255, (pages, PT * ROW), generator=g, device="cuda", dtype=torch.uint8)
             if fp8 else torch.randn(pages, PT * ROW, generator=g, device="cuda").bfloat16()
             for _ in range(layers)]
    host = [s.cpu().view(torch.uint8 if fp8 else torch.int16).numpy() for s in slabs]
    each = rng.integers(0, new + 1, len(lens))
    t, c = _ints(wide), _ints(counts)
    for n_new in ([new] * len(lens), each):
        want, wide, counts, served = oracle.pages_reserve(host, wide, lens, n_new, counts)
        status = _ints([0])
        given = new if isinstance(n_new, list) else _ints(n_new)
        api.mla_pages_reserve(slabs, t, _ints(lens), given, c, status=status)
        assert int(status.item()) == (0 if all(served) else 35)
        assert np.array_equal(t.cpu().numpy(), wide)
        assert np.array_equal(c.cpu().numpy(), counts)
        for s, w in zip(slabs, want):
            assert np.array_equal(s.cpu().view(torch.uint8 if fp8 else torch.int16).numpy(), w)
        host = want


@pytest.mark.parametrize("pages,first", [(16_384, 0), (16_385, 16_380), (70_001, 69_000),
                                         (70_001, 10), (100_000, 40_000)])
def test_free_pages_are_found_in_ascending_order(pages, first):
    """Pools of several sweeps; free pages here and there from `first` on.  (Nothing is
    copied, so the pool can stand in for a larger one: one page, expanded.)"""
    rng = np.random.default_rng(pages + first)
    counts = np.ones(pages, np.int32)
    free = np.sort(first + rng.choice(pages - first, min(700, pages - first), replace=False))
    counts[free] = 0
    lens = rng.integers(0, 3, 300) * PT
    table = np.tile(np.arange(9, dtype=np.int32), (300, 1))
    need = [int(x) for x in rng.integers(0, 4, 300)]
    slab = torch.zeros(1, PT * ROW, dtype=torch.uint8, device="cuda")
    d = dict(t=_ints(table), c=_ints(counts))
    lib = api._native.lib()
    import ctypes
    work = torch.empty(lib.mla_pages_workspace_size(300), dtype=torch.uint8, device="cuda")
    status, new, at = _ints([0]), _ints([n * PT for n in need]), _ints(lens)
    rc = lib.mla_pages_reserve(1, (ctypes.c_void_p * 1)(slab.data_ptr()), 1, pages, PT * ROW,
                               d["t"].data_ptr(), 9, 9, at.data_ptr(), 300, 0, new.data_ptr(),
                               d["c"].data_ptr(), work.data_ptr(), work.numel(),
                               status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    _, want, c, served = oracle.pages_reserve([], table, lens, [n * PT for n in need], counts)
    assert np.array_equal(d["t"].cpu().numpy(), want)
    assert np.array_equal(d["c"].cpu().numpy(), c)
    assert int(status.item()) == (0 if all(served) else 35)


def test_many_rows_part_from_one_page():
    """1,024 continuations of one history: all but the last copy its last page."""
    rows, pages = 1024, 1100
    table = np.zeros((rows, 2), np.int32)
    counts = np.zeros(pages, np.int32)
    counts[0] = rows
    counts[5:9] = 1
    slab = torch.zeros(pages, PT * ROW, dtype=torch.uint8, device="cuda")
    slab[0, :7 * ROW] = torch.arange(7 * ROW, device="cuda").to(torch.uint8)
    t, c = _ints(table), _ints(counts)
    api.mla_pages_reserve([slab], t, _ints([7] * rows), 1, c)
    ids = t[:, 0].cpu().numpy()
    assert ids[-1] == 0 and len(set(ids)) == rows and not set(ids) & {5, 6, 7, 8}
    assert np.array_equal(np.sort(ids[:-1]), ids[:-1])
    assert c.cpu().numpy()[ids].tolist() == [1] * rows
    assert bool((slab[t[:, 0].long(), :7 * ROW] == slab[0, :7 * ROW]).all())
    assert not slab[t[:-1, 0].long(), 7 * ROW:].any()


def test_what_does_not_fit_is_reported_and_left():
    slab = torch.zeros(8, PT * ROW, dtype=torch.bfloat16, device="cuda")

    def fork(table, lens, parents, out_lens=(0, 0), cols=3):
        c, st = _ints([2, 2, 2, 2, 0, 0, 0, 0]), _ints([0])
        out, n = _ints(np.full((2, cols), 3)), _ints(out_lens)
        api.mla_pages_fork(_ints(table), _ints(lens), _ints(parents), c, out, n, status=st)
        return int(st.item()), out.tolist(), n.tolist(), c.tolist()

    two = [[0, 1], [2, 3]]
    assert fork(two, [PT + 1, PT], [1, 0]) == (0, [[2, 3, 3], [0, 1, 3]], [PT, PT + 1],
                                              [3, 3, 3, 2, 0, 0, 0, 0])
    assert fork(two, [PT, PT], [2, -1])[:3] == (36, [[3] * 3, [3] * 3], [0, 0])
    assert fork(two, [2 * PT + 1, -5], [0, 1])[:3] == (33, [[3] * 3, [3] * 3], [0, 0])
    assert fork(two, [2 * PT, 0], [0, 1], cols=1)[:3] == (33, [[3], [3]], [0, 0])
    assert fork([[0, 8], [-1, 1]], [2 * PT, 1], [0, 1])[::3] == (33, [3, 2, 2, 2, 0, 0, 0, 0])
    # an out row that says it holds a page which no one holds
    st = _ints([0])
    c, n, out = _ints([1, 0, 0, 0, 0, 0, 0, 0]), _ints([1]), _ints([[4]])
    api.mla_pages_fork(_ints([[0]]), _ints([1]), _ints([0]), c, out, n, status=st)
    assert int(st.item()) == 37 and c.tolist() == [2] + [0] * 7

    def reserve(table, lens, new, counts, cols=3):
        c, st = _ints(counts), _ints([0])
        t = _ints(table)
        api.mla_pages_reserve([slab], t, _ints(lens), new, c, status=st)
        return int(st.item()), t.tolist(), c.tolist()

    full = [1] * 8
    assert reserve([[0, 9, 9]], [PT], 1, full) == (35, [[0, 9, 9]], full)
    assert reserve([[0, 9, 9]], [PT - 1], 1, full) == (0, [[0, 9, 9]], full)
    assert reserve([[0, 9, 9]], [5], 3 * PT, [1] + [0] * 7)[::2] == (33, [1] + [0] * 7)
    assert reserve([[0, 9, 9]], [-1], 1, full)[0] == 32
    assert reserve([[0, 9, 9]], [1], _ints([-1]), full)[0] == 32
    assert reserve([[8, 9, 9]], [1], 1, full)[0] == 33
    assert reserve([[0, 9, 9]], [1], 1, [0] * 8)[0] == 37
    # the first row takes the only page, the second gets none, the third needs none
    some = [1, 1, 1, 1, 1, 1, 1, 0]
    assert reserve([[0, 9], [1, 9], [2, 9]], [PT, PT, 3], 1, some) == \
        (35, [[0, 7], [1, 9], [2, 9]], full)
    assert reserve([[0, 9]], [PT], 0, some) == (0, [[0, 9]], some)


def test_refusals():
    t, n, c = _ints([[0, 1]]), _ints([5]), _ints([1, 1, 0, 0])
    out, m, p = _ints([[0, 0]]), _ints([0]), _ints([0])
    slab = torch.zeros(4, PT * ROW, dtype=torch.bfloat16, device="cuda")
    both = torch.zeros(4, 4, dtype=torch.int32, device="cuda")
    pair = torch.zeros(3, dtype=torch.int32, device="cuda")
    bad = [
        lambda: api.mla_pages_fork(t, n, p, c, t, m), lambda: api.mla_pages_fork(t, n, p, c, out, n),
        lambda: api.mla_pages_fork(both[:3], pair, pair.clone(), c, both[1:], pair.clone()),
        lambda: api.mla_pages_fork(t, pair[:1], p, c, out, pair[:1]),
        lambda: api.mla_pages_fork(t.long(), n, p, c, out, m),
        lambda: api.mla_pages_fork(t.cpu(), n, p, c, out, m),
        lambda: api.mla_pages_fork(t, n, p, c.float(), out, m),
        lambda: api.mla_pages_fork(t, n, p, c[::2], out, m),
        lambda: api.mla_pages_fork(t, n, p, c, out, m, status=torch.zeros(1, device="cuda")),
        lambda: api.mla_pages_free(t, n[:0], c), lambda: api.mla_pages_free(t, n, c.long()),
        lambda: api.mla_pages_reserve([], t, n, 1, c), lambda: api.mla_pages_reserve(slab, t, n, 1, c),
        lambda: api.mla_pages_reserve([slab], t, n, -1, c),
        lambda: api.mla_pages_reserve([slab], t, n, 1, c[:3]),
        lambda: api.mla_pages_reserve([slab, slab[:2]], t, n, 1, c),
        lambda: api.mla_pages_reserve([slab], t, n, _ints([1, 2]), c),
        lambda: api.mla_pages_reserve([slab], t, n, 1, c,
                                      workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
    ]
    for call in bad:
        with pytest.raises((ValueError, RuntimeError)):
            call()
    # rows of one wider table, side by side, are not refused
    api.mla_pages_fork(both[:2, :2], pair[:2], _ints([0, 1]), c, both[:2, 2:], _ints([0, 0]))


def test_views_streams_and_graph_replay():
    """A search's step in a graph: tables that are views, lengths that change in place."""
    pages = 64
    wide = torch.full((4, 11), -1, dtype=torch.int32, device="cuda")
    a, b = wide[:, :5], wide[:, 6:]
    a[:, 0] = 3
    lens, out_lens = _ints([100] * 4), _ints([0] * 4)
    counts = torch.zeros(pages, dtype=torch.int32, device="cuda")
    counts[3] = 4
    parents = _ints([0, 0, 2, 3])
    slab = torch.zeros(pages, PT * ROW, dtype=torch.bfloat16, device="cuda")
    slab[3, :100 * ROW] = 1
    keep = [x.clone() for x in (wide, lens, out_lens, counts)]

    def step(stream=None):
        api.mla_pages_fork(a, lens, parents, counts, b, out_lens, stream=stream)
        api.mla_pages_free(a, lens, counts, stream=stream)
        api.mla_pages_reserve([slab], b, out_lens, 1, counts, stream=stream)

    step()
    want = [x.clone() for x in (wide, lens, out_lens, counts)]
    assert want[0][:, 6].tolist() == [0, 1, 2, 3] and want[1].tolist() == [0] * 4
    assert bool((slab[:4, :100 * ROW] == 1).all())
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    for run in ("side", "graph"):
        if run == "graph":
            with torch.cuda.graph(graph):
                step()
        for _ in range(2):
            for x, k in zip((wide, lens, out_lens, counts), keep):
                x.copy_(k)
            if run == "graph":
                graph.replay()
            else:
                side.wait_stream(torch.cuda.current_stream())
                step(side)
                side.synchronize()
            assert all(torch.equal(x, w) for x, w in zip((wide, lens, out_lens, counts), want))
