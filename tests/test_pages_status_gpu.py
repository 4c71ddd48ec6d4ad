"""What forks and releases of pages do with lengths and counts that cannot be right."""
import numpy as np
import pytest
import torch

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
