"""What forks and releases of pages do with lengths and counts that cannot be right."""
import numpy as np
import pytest
import torch

import oracle
from paged_latent_attention_gb300 import api

pytestmark = pytest.mark.gpu

PT = 1536


def _ints(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device="cuda")


def _fork(table, lens, parents, counts, out, out_lens):
    c, st, o, n = _ints(counts), _ints([0]), _ints(out), _ints(out_lens)
    api.mla_pages_fork(_ints(table), _ints(lens), _ints(parents), c, o, n, status=st)
    return int(st.item()), o.tolist(), n.tolist(), c.tolist()


def test_a_negative_length_is_reported_and_the_row_left():
    two, out = [[0, 1], [2, 3]], [[4, 5], [6, 7]]
    counts = [1] * 8
    # of the source row
    assert _fork(two, [PT, -1], [1, 0], counts, out, [2 * PT, 9]) == \
        (32, [[4, 5], [0, 7]], [2 * PT, PT], [2, 1, 1, 1, 1, 1, 0, 1])
    assert _fork(two, [-2 ** 31, -1], [1, 0], counts, out, [0, 9]) == (32, out, [0, 9], counts)
    # of the out row
    assert _fork(two, [PT, 5], [1, 0], counts, out, [-7, 9]) == \
        (32, [[4, 5], [0, 7]], [-7, PT], [2, 1, 1, 1, 1, 1, 0, 1])
    assert _fork(two, [PT, 5], [-1, -1], counts, out, [-7, 9]) == \
        (32, out, [-7, 0], [1, 1, 1, 1, 1, 1, 0, 1])
    n, c, st = _ints([-3, 5]), _ints(counts), _ints([0])
    api.mla_pages_free(_ints(two), n, c, status=st)
    assert int(st.item()) == 32 and n.tolist() == [-3, 0] and c.tolist() == [1, 1, 0] + [1] * 5


def test_of_several_codes_the_largest_stays():
    rows = 600
    table = np.zeros((rows, 2), np.int32)
    lens = np.where(np.arange(rows) % 3 == 0, -1, 1)
    parents = np.where(np.arange(rows) % 3 == 1, rows + 5, np.arange(rows))
    for _ in range(20):
        got = _fork(table, lens, parents, [rows] + [1] * 3, np.zeros((rows, 2)), np.zeros(rows))
        assert got[0] == 36
        st, n = _ints([0]), _ints(np.where(np.arange(rows) % 2 == 0, -1, 3 * PT))
        api.mla_pages_free(_ints(table), n, _ints([2 * rows]), status=st)
        assert int(st.item()) == 33


@pytest.mark.parametrize("rows", [2, 8, 10, 64, 66, 1000])
def test_counts_of_an_under_counted_fork_do_not_depend_on_the_order_of_rows(rows):
    """A count becomes what was counted, plus what is taken, less what is given up, or 0."""
    rng = np.random.default_rng(rows)
    table, out = rng.permutation(rows)[:, None], rng.permutation(rows)[:, None]
    parents = rng.permutation(rows)
    half = rows // 2
    twice = np.concatenate([np.arange(half), np.arange(half)])[:, None]
    to = np.where(np.arange(rows) < half, np.arange(rows), -1)
    for have in (0, 1, 2):
        for _ in range(10):
            # each page loses a holder and gains one
            status, o, n, c = _fork(table, [1] * rows, parents, [have] * rows, out, [1] * rows)
            assert c == [have] * rows and status == 0
            assert o == table[parents].tolist() and n == [1] * rows
            # each page loses two and gains one
            status, _, _, c = _fork(np.roll(np.arange(half), 1)[:, None], [1] * half, to, [have] * half,
                                    twice, [1] * rows)
            assert c == [max(0, have - 1)] * half and status == (0 if have else 37)


@pytest.mark.parametrize("rows", [3, 8, 9, 57, 64, 65])
def test_forks_around_the_sizes_of_a_cluster(rows):
    """Rows of more columns than threads, some left as they are, some emptied."""
    rng = np.random.default_rng(rows)
    cols, pages = 300, 400_000
    table = rng.permutation(pages)[:rows * cols].reshape(rows, cols)
    lens = rng.integers(0, cols * PT + 1, rows)
    parents = rng.integers(-1, rows, rows)
    counts = np.zeros(pages, np.int64)
    out, n = np.full((rows, cols), 7), np.zeros(rows, np.int64)
    for r in range(rows):
        counts[table[r, :-(-lens[r] // PT)]] += 1
    d = [_ints(x) for x in (table, lens, counts, out, n)]
    st = _ints([0])
    for _ in range(3):
        out, n, counts = oracle.pages_fork(table, lens, parents, counts, out, n)
        api.mla_pages_fork(d[0], d[1], _ints(parents), d[2], d[3], d[4], status=st)
        for got, want in zip(d[2:], (counts, out, n)):
            assert np.array_equal(got.cpu().numpy(), want)
        parents = rng.integers(-1, rows, rows)
    assert int(st.item()) == 0
