"""Which rows mla_pages_reserve had room for, row by row against the oracle."""
import numpy as np
import pytest
import torch

import oracle
from paged_latent_attention_gb300 import api

pytestmark = pytest.mark.gpu

PT, ROW = 1536, 576


def _ints(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device="cuda")


def _slab(pages):
    return torch.zeros(pages, PT * ROW, dtype=torch.uint8, device="cuda")


def test_rows_that_share_a_page_without_free_ones():
    """The first holder cannot leave the page, so the second must not write to it."""
    slab = _slab(4)

    def reserve(table, lens, new, counts):
        t, c, st, got = _ints(table), _ints(counts), _ints([0]), _ints([77] * len(lens))
        assert api.mla_pages_reserve([slab], t, _ints(lens), new, c, status=st, granted=got) is t
        return int(st.item()), got.tolist(), t.tolist(), c.tolist()

    two = [[0, 9], [0, 9]]
    assert reserve(two, [7, 7], 1, [2, 1, 1, 1]) == (35, [0, 0], two, [2, 1, 1, 1])
    assert reserve(two, [9, 5], 1, [2, 1, 1, 1]) == (35, [0, 0], two, [2, 1, 1, 1])
    assert reserve(two, [7, 7], 3, [2, 1, 0, 1]) == (0, [3, 3], [[2, 9], [0, 9]], [1, 1, 1, 1])
    # a row that gets nothing new leaves the other a holder to part from
    assert reserve(two, [7, 7], _ints([0, 1]), [2, 1, 1, 1]) == (35, [0, 0], two, [2, 1, 1, 1])
    assert reserve(two, [7, 7], _ints([0, 4]), [2, 1, 0, 1]) == (0, [0, 4], [[0, 9], [2, 9]], [1, 1, 1, 1])
    # the first of three leaves, the second finds no page, the third then shares with it
    three = [[0, 9]] * 3
    assert reserve(three, [7] * 3, 1, [3, 1, 0, 1]) == \
        (35, [1, 0, 0], [[2, 9], [0, 9], [0, 9]], [2, 1, 1, 1])
    # an earlier row is refused for another page: a later one alone on its own goes on
    assert reserve([[1, 9], [0, 9], [2, 9]], [PT, 7, 7], 1, [1, 1, 1, 1])[:2] == (35, [0, 1, 1])
    # lengths and pages out of range
    assert reserve([[0, 9], [1, 9], [7, 9]], [-1, 2 * PT, 5], 1, [1, 1, 1, 1])[1] == [0, 0, 0]
    assert reserve([[0, 9], [1, 9]], [5, 5], _ints([-2, 2]), [1, 1, 1, 1])[:2] == (32, [0, 2])


@pytest.mark.parametrize("seed", range(12))
def test_matches_the_oracle_row_by_row(seed):
    """Rows in families that share partly filled pages, and fewer free pages than they need."""
    rng = np.random.default_rng(seed)
    rows, pages = int(rng.integers(2, 1025 if seed % 3 == 0 else 40)), 3000
    ids = rng.permutation(pages)
    table = np.full((rows, 6), 9999, np.int64)
    lens = np.zeros(rows, np.int64)
    counts = np.zeros(pages, np.int64)
    at = 0
    for r in range(rows):
        old = int(rng.integers(0, r)) if r and rng.random() < 0.7 else -1
        if old >= 0:
            lens[r], table[r] = lens[old], table[old]
        else:
            lens[r] = rng.integers(0, 2 * PT)
            n = -(-int(lens[r]) // PT)
            table[r, :n] = ids[at:at + n]
            at += n
        for c in range(-(-int(lens[r]) // PT)):
            counts[table[r, c]] += 1
    new = rng.integers(0, 2 * PT, rows) * (rng.random(rows) < 0.5) + (rng.random(rows) < 0.7)
    order = rng.permutation(rows)
    table, lens = table[order], lens[order]
    spare = ids[at:]
    counts[spare[int(rng.integers(0, max(2, rows))):]] = 1
    t, c, st, got = _ints(table), _ints(counts), _ints([0]), _ints(new)
    slab = torch.empty(pages, PT * ROW, dtype=torch.uint8, device="cuda")
    _, want, left, served = oracle.pages_reserve([], table, lens, new, counts)
    api.mla_pages_reserve([slab], t, _ints(lens), got, c, status=st, granted=got)
    assert got.tolist() == [int(n) if ok else 0 for n, ok in zip(new, served)]
    assert int(st.item()) == (0 if all(served) else 35)
    assert np.array_equal(t.cpu().numpy(), want) and np.array_equal(c.cpu().numpy(), left)


def test_a_search_goes_on_without_the_rows_that_have_no_room():
    """README's step with a pool that runs out: no row's tokens are overwritten."""
    pages, R = 5, 4
    slab = torch.zeros(pages, PT * ROW, dtype=torch.bfloat16, device="cuda")
    table = _ints([[0, 9], [0, 9], [0, 9], [1, 9]])
    lens, counts = _ints([PT - 2, PT - 2, PT - 2, 10]), _ints([3, 1, 1, 0, 1])
    slab.view(pages, PT, ROW)[0, :PT - 2] = 1.0
    slab.view(pages, PT, ROW)[1, :10] = 2.0
    status, granted = _ints([0]), _ints([0] * R)
    have = [[1.0] * (PT - 2)] * 3 + [[2.0] * 10]
    for step in range(4):
        api.mla_pages_reserve([slab], table, lens, 1, counts, granted=granted, status=status)
        lens += granted
        x = (torch.arange(R, device="cuda") + 10.0 * (step + 1)).bfloat16()[:, None]
        api.mla_kv_append(x.expand(R, 512).contiguous(), x.expand(R, 64).contiguous(), slab, table,
                          lens * granted, 1)
        have = [h + [float(x[r])] if granted[r] else h for r, h in enumerate(have)]
        assert lens.tolist() == [len(h) for h in have]
        for r, h in enumerate(have):
            t = torch.arange(len(h), device="cuda")
            got = slab.view(pages, PT, ROW)[table[r].long()[t // PT], t % PT]
            assert torch.equal(got[:, 0].float().cpu(), torch.tensor(h)) and bool((got == got[:, :1]).all())
    assert int(status.item()) == 35 and lens.tolist() == [PT, PT - 2, PT - 2, 14]


def test_a_row_on_a_page_without_holders_is_left_alone():
    """Its page looks free, and may go to another row."""
    slab = _slab(4)
    for table, lens, new, counts in (
            ([[0, 9], [1, 9]], [7, PT], [1, 1], [0, 1, 1, 1]),
            ([[2, 9], [1, 9]], [PT - 1, 8], [PT, 1], [1, 1, 0, 0]),
            ([[3, 9], [3, 9], [0, 9]], [5, 6, 7], [1, 1, 1], [2, 1, 0, 0])):
        t, c, st, got = _ints(table), _ints(counts), _ints([0]), _ints([0] * len(lens))
        _, want, left, served = oracle.pages_reserve([], table, lens, new, counts)
        api.mla_pages_reserve([slab], t, _ints(lens), _ints(new), c, status=st, granted=got)
        assert int(st.item()) == 37 and not served[0]
        assert got.tolist() == [n if ok else 0 for n, ok in zip(new, served)]
        assert np.array_equal(t.cpu().numpy(), want) and np.array_equal(c.cpu().numpy(), left)
