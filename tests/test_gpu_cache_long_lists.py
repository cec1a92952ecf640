"""GPU tests of resizes of long lists: past the entries that look through each other, past the workgroups of a launch,
and past the 2^24 workgroups of 256 threads that a grid cannot hold."""
import random

import pytest
import torch

from copy_reduce_amd import TB_CACHE_RANGE, TB_CACHE_TWICE
from gpu_util import note, require_gpu
from test_gpu_cache import ints, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [2047, 4096, 4097, 9000, 70001])
def test_long_lists(n):
    """Rows of up to 3 pages that come, change and go, with padding, rows and lengths out of range and rows listed again."""
    note(f"paged cache, resize of {n} entries")
    r = random.Random(n)
    c, m = make(pages=3 * n // 2, pt=2, seqs=n, width=3, heads=1, dim=8)
    for step in range(3):
        seqs = r.sample(range(n), n)
        lens = [r.randrange(m.MP * m.pt + 1) if r.random() < 0.4 else 0 for _ in seqs]
        if step:
            for _ in range(n // 50):
                seqs[r.randrange(n)] = r.choice([-1, n, seqs[r.randrange(n)], seqs[0], seqs[-1]])
                lens[r.randrange(n)] = r.choice([-1, m.MP * m.pt + 1])
        c.resize(ints(seqs), ints(lens)), m.resize(seqs, lens)
        m.check(c, f"step {step}")
        flags = c.flags(clear=True)
        m.flags = 0
        assert not step or flags & (TB_CACHE_RANGE | TB_CACHE_TWICE) == TB_CACHE_RANGE | TB_CACHE_TWICE
    c.resize(ints(list(range(n))), ints([0] * n)), m.resize(list(range(n)), [0] * n)
    m.check(c, "all freed")
    assert int(c.counts[0]) == m.P and c.flags() == 0


@pytest.mark.parametrize("n", [(1 << 24) - 1, (1 << 24) + 5])
def test_lists_past_a_grid(n):
    """As many entries as rows: those of every 40,000th row take a page, and go again."""
    note(f"paged cache, resize of {n} entries")
    require_gpu()
    from copy_reduce_amd.torch_api import PagedCache
    every = 40000
    c = PagedCache(torch.zeros(2, 500, 1, 1, 8, dtype=torch.bfloat16, device="cuda"), 1, n, 1)
    seqs = torch.arange(n, dtype=torch.int32, device="cuda")
    lens = (seqs % every == every - 1).to(torch.int32)
    lens[-1] = 1
    seqs[0] = n - 1                                    # the last row comes first, to no tokens: its own entry is one too many
    c.resize(seqs, lens)
    assert c.flags(clear=True) == TB_CACHE_TWICE
    took = n // every - (n % every == 0)
    want = torch.zeros(n, dtype=torch.int32, device="cuda")
    want[every - 1::every] = 1
    want[-1] = 0
    assert torch.equal(c.lens, want) and int(c.counts[0]) == 500 - took
    assert c.table[every - 1::every, 0].tolist()[:took] == list(range(took))
    assert c.refs.tolist() == [1] * took + [0] * (500 - took)
    c.resize(torch.arange(n, dtype=torch.int32, device="cuda"), torch.zeros_like(lens))
    assert c.flags() == 0 and int(c.counts[0]) == 500 and not c.lens.any() and not c.refs.any()
    assert c.free_list.tolist() == list(range(499, -1, -1))
