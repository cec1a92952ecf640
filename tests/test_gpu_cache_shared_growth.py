"""GPU tests of rows that are cut back into a page that another row refers to: they cannot grow in it (their tokens
would be written to the other row as well, or not at all), a fork of them can."""
import random

import pytest
import torch

from cache_model import Model, attention
from copy_reduce_amd import TB_CACHE_RANGE, TB_CACHE_SHARED
from gpu_util import note, require_gpu
from test_gpu_cache import ints, make

pytestmark = pytest.mark.gpu


def resize(m, seqs, lens):
    """The model's resize without the entries that would grow in a shared page, which raise the flag."""
    after, seen = list(m.refs), set()
    for q, n in zip(seqs, lens):
        if 0 <= q < m.S and q not in seen:
            seen.add(q)
            if 0 <= n <= m.MP * m.pt:
                for page in m.table[q][m.npg(n):m.npg(m.lens[q])]:
                    after[page] -= 1
    seen, kept = set(), []
    for q, n in zip(seqs, lens):
        if 0 <= q < m.S and q not in seen:
            seen.add(q)
            had = m.lens[q]
            if had < n <= m.MP * m.pt and had % m.pt and after[m.table[q][had // m.pt]] > 1:
                m.flags |= TB_CACHE_SHARED
                kept.append((q, had))     # stands in the list: a later entry of the row is still one too many
                continue
        kept.append((q, n))
    m.resize(*[list(x) for x in zip(*kept)] if kept else ([], []))


def both(c, m, name, *args):
    getattr(c, name)(*[ints(a) if isinstance(a, list) else a.cuda() for a in args])
    resize(m, *args) if name == "resize" else getattr(m, name)(*args)
    m.check(c, f"{name} {[a for a in args if isinstance(a, list)]}")


def attends_as_defined(c, m, seqs, seed):
    from copy_reduce_amd.torch_api import tree_attention
    g = torch.Generator().manual_seed(seed)
    q, k, v = [torch.randn(len(seqs), 1, h, 64, generator=g).to(torch.bfloat16) for h in (4, 2, 2)]
    got, _ = tree_attention(q.cuda(), k.cuda(), v.cuda(), c, 0, ints(seqs))
    out, _, a, s, _ = attention(m, 0, q, k, v, seqs)
    # a half step of the result and of each weight, scores of 64 products in fp32, and sums of few terms (far below 2^-16)
    tol = out.abs() * 2 ** -8 + a * (2 ** -8 + 2 * (2 * 64 + 8) * 2 ** -24 * s + 2 ** -16)[..., None]
    assert bool(((got.double().cpu() - out).abs() <= tol).all())


def values(c, n, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(len(c.pools), n, c.heads, c.head_dim, generator=g).to(c.dtype)


@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("wide", [False, True], ids=["one workgroup", "three launches"])
def test_cut_back_into_a_shared_page(layout, wide):
    """Fork, cut back, grow, append, attend; then the same by way of a fork."""
    note(f"paged cache, growth in a shared page, {layout}, wide {wide}")
    pt = 4
    c, m = make(pages=40, pt=pt, seqs=6, width=600 if wide else 9, heads=2, dim=64, layout=layout)
    both(c, m, "resize", [0], [8])
    both(c, m, "append", values(c, 8, 1), [0] * 8, list(range(8)))
    both(c, m, "fork", [0], [1])
    both(c, m, "resize", [1], [6])                       # the child goes back to its sixth token
    both(c, m, "resize", [1, 0], [7, 9])                 # the parent has a page of its own to go on with
    assert c.lens.tolist()[:2] == [9, 6] and c.flags(clear=True) == TB_CACHE_SHARED
    m.flags = 0
    both(c, m, "append", values(c, 2, 2), [1, 0], [6, 8])
    assert c.flags(clear=True) == TB_CACHE_RANGE         # the child has no seventh token
    m.flags = 0
    attends_as_defined(c, m, [1, 0], 3)

    both(c, m, "fork", [1], [2])                         # the way on: a row whose sixth token is its own
    both(c, m, "resize", [1, 2], [0, 11])
    both(c, m, "append", values(c, 5, 4), [2] * 5, list(range(6, 11)))
    attends_as_defined(c, m, [2, 0], 5)
    assert c.flags() == 0


@pytest.mark.parametrize("wide", [False, True], ids=["one workgroup", "three launches"])
def test_who_holds_the_page_after_the_call_decides(wide):
    """Both holders grow: neither does.  One goes in the same call: the other may.  The same length is no growth."""
    note(f"paged cache, growth in a shared page, both holders, wide {wide}")
    c, m = make(pages=40, pt=4, seqs=6, width=600 if wide else 9)
    both(c, m, "resize", [0], [12])
    both(c, m, "fork", [0, 0], [1, 2])
    both(c, m, "resize", [0, 1, 2], [6, 6, 6])
    both(c, m, "resize", [0, 1, 2], [6, 5, 5])           # shorter and the same: no flag
    assert c.flags() == 0
    both(c, m, "resize", [0, 1, 2], [7, 30, 6])
    assert c.flags(clear=True) == TB_CACHE_SHARED and c.lens.tolist()[:3] == [6, 5, 5]
    m.flags = 0
    both(c, m, "resize", [2, 1, 0], [0, 30, 0])          # only the row that grows is left
    assert c.flags() == 0 and c.lens.tolist()[:3] == [0, 30, 0]
    both(c, m, "resize", [1], [0])
    assert int(c.counts[0]) == m.P


@pytest.mark.parametrize("seed", range(1, 13))
def test_random_forks_cuts_and_growth(seed):
    """Every resize that the model allows, and no other: lists of 1 to 60 entries over caches with room to grow."""
    note(f"paged cache, random forks, cuts and growth, seed {seed}")
    r = random.Random(seed)
    c, m = make(pages=r.choice([60, 300]), pt=r.choice([2, 3, 8]), seqs=r.choice([4, 20, 60]), width=r.choice([5, 9, 700]))
    refused = 0
    for step in range(60):
        n = r.randrange(1, m.S + 1)
        seqs = r.sample(range(m.S), n)
        if r.random() < 0.35:
            live = [q for q in range(m.S) if m.lens[q]] or [0]
            empty = [q for q in range(m.S) if not m.lens[q]][:n]
            if empty:
                both(c, m, "fork", [r.choice(live) for _ in empty], empty)
            continue
        most = min(m.MP, 9) * m.pt
        lens = [max(0, min(most, r.choice([0, m.lens[q] - r.randrange(6), m.lens[q] + r.randrange(6), r.randrange(most + 1)]))) for q in seqs]
        m.flags = 0
        c.counts[1] = 0
        both(c, m, "resize", seqs, lens)
        refused += bool(m.flags & TB_CACHE_SHARED)
    assert refused
