"""Histories that have outgrown their rows of weights are reported by the selection."""
import numpy as np
import pytest
import torch

import oracle
from paged_latent_attention_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,keep,recent", [(100, 30, 4), (100, 100, 7), (5000, 900, 60),
                                                (500_000, 1000, 64)])
@pytest.mark.parametrize("over", [0, 1, 2000])
def test_a_history_past_its_row_is_reported(tokens, keep, recent, over):
    """`over` tokens have no weight: they cannot stay, and the caller is told so."""
    mass = torch.rand(2, tokens, device="cuda")
    lens = [tokens // 3, tokens + over]
    dev = torch.as_tensor(np.asarray(lens, dtype=np.int32), device="cuda")
    for before in (0, 7):
        status = torch.full((1,), before, dtype=torch.int32, device="cuda")
        kept, n = api.mla_evict_select(mass, dev, keep, sink=2, recent=recent, status=status)
        assert int(status.item()) == (34 if over else before)
        want = oracle.evict_select(mass.cpu().numpy(), lens, keep, 2, recent)
        assert [kept[r, : len(k)].tolist() for r, k in enumerate(want)] == want
        assert n.tolist() == [len(k) for k in want]
    for status in (torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(ValueError):
            api.mla_evict_select(mass, dev, keep, status=status)


def test_lengths_are_not_overwritten():
    """Every CTA of a request reads its length while one of them writes kept_lens: the
    two in one place would race, and the compaction needs the lengths as they were."""
    mass = torch.rand(3, 5000, device="cuda")
    both = torch.tensor([5000, 4000, 10, 7], dtype=torch.int32, device="cuda")
    for kept_lens in (both[:3], both[1:]):
        with pytest.raises(ValueError):
            api.mla_evict_select(mass, both[:3], 900, kept_lens=kept_lens)
    apart = torch.tensor([5000, 4000, 10, 0, 0, 0], dtype=torch.int32, device="cuda")
    _, n = api.mla_evict_select(mass, apart[:3], 900, kept_lens=apart[3:])
    assert apart.tolist() == [5000, 4000, 10, 900, 900, 10] and n.data_ptr() == apart[3:].data_ptr()


def test_threads_agree_on_the_form():
    """The form of a selection goes by what the device holds at once, asked by whichever
    thread comes first: all get the same size and the same tokens."""
    from concurrent.futures import ThreadPoolExecutor

    shapes = [(1, 300), (3, 60_000), (2, 500_000), (1, 1_000_000), (40, 20_000)]

    def sizes(_):
        return [api.allocate_evict_workspace(*shape).numel() for shape in shapes]

    mass = torch.rand(2, 500_000, device="cuda")
    lens = torch.tensor([500_000, 400_000], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()

    def select(_):
        with torch.cuda.stream(torch.cuda.Stream()):
            kept, _ = api.mla_evict_select(mass, lens, 40_000, recent=10)
            torch.cuda.current_stream().synchronize()
            return kept

    with ThreadPoolExecutor(8) as pool:
        got = list(pool.map(sizes, range(64)))
        kept = list(pool.map(select, range(16)))
    assert all(s == got[0] for s in got) and got[0][2] > 0 and got[0][0] == 0
    assert all(torch.equal(k, kept[0]) for k in kept)
