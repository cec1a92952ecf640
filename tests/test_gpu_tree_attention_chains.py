"""GPU tests of tb_tree_attention over chains and trees of hundreds to thousands of nodes (a prompt's chunk attending
over the cache), and of page numbers out of range.  Bounds as in test_gpu_tree_attention.py."""
import math

import pytest
import torch

from gpu_util import note
from test_gpu_tree_attention import compare, inputs, ints, setup, tree_mask

pytestmark = pytest.mark.gpu


def definition(m, q, k, v, seqs, mask, count):
    """As cache_model.attention, all nodes of a head at once."""
    b, t, hq, d = q.shape
    hk = k.shape[2]
    g = hq // hk
    out, a = torch.zeros(b, t, hq, d, dtype=torch.float64), torch.zeros(b, t, hq, d, dtype=torch.float64)
    lse, s, big = [torch.full((b, t, hq), x, dtype=torch.float64) for x in (-math.inf, 0.0, 0.0)]
    for i, row in enumerate(seqs):
        c = t if count is None else count[i]
        if mask is None:
            sees = torch.ones(c, c, dtype=torch.bool).tril()
        else:
            u = torch.arange(c)
            sees = (mask[i, :c][:, u // 64] >> (u % 64) & 1).bool()
        for h in range(hk):
            key = torch.cat([m.context(0, row, h), k[i, :c, h].double()])
            val = torch.cat([m.context(1, row, h), v[i, :c, h].double()])
            all_see = torch.cat([torch.ones(c, len(key) - c, dtype=torch.bool), sees], 1)
            for j in range(h * g, h * g + g):
                qq = q[i, :c, j].double()
                x = (qq @ key.T.contiguous() / math.sqrt(d)).masked_fill(~all_see, -math.inf)
                z = torch.logsumexp(x, 1)
                w = torch.exp(x - z[:, None])
                out[i, :c, j], a[i, :c, j], lse[i, :c, j] = w @ val, w @ val.abs(), z
                s[i, :c, j] = (qq.abs() @ key.abs().T.contiguous() / math.sqrt(d)).masked_fill(~all_see, 0).amax(1)
                big[i, :c, j] = torch.where(all_see, val.abs().amax(1), 0.0).amax(1)
    return out, lse, a, s, big


def run(c, m, x, seqs, mask=None, count=None, what=""):
    from copy_reduce_amd.torch_api import tree_attention
    got = tree_attention(*[t.cuda() for t in x], c, 0, ints(seqs), mask=None if mask is None else mask.cuda(),
                         nodes=None if count is None else ints(count))
    compare(got, definition(m, *x, seqs, mask, count), max(m.lens) + x[0].shape[1], x[0].shape[3], x[0].dtype, what)


@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("dim,group", [(64, 1), (96, 3), (128, 4), (256, 2)])
@pytest.mark.parametrize("nodes", [257, 1000])
def test_chunks_of_a_prompt(nodes, dim, group, dtype, room):
    note(f"tree attention, chains of {nodes}, {group} rows a node, dim {dim} {dtype} room {room}")
    c, m, g = setup([0, 37, 700], heads=2, dim=dim, dtype=dtype, seed=nodes + dim, room=room)
    run(c, m, inputs(g, 3, nodes, 2 * group, 2, dim, dtype), [2, 0, 1], count=[nodes, nodes - 1, nodes // 2], what="chains")


@pytest.mark.parametrize("lens", [[0], [2000]])
def test_longest_chain(lens):
    note(f"tree attention, a chain of 4,096 over {lens}")
    c, m, g = setup(lens, heads=2, dim=128, seed=1)
    run(c, m, inputs(g, 1, 4096, 4, 2, 128, torch.bfloat16), [0], what="the longest chain")


@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])
def test_wide_trees_by_mask(room):
    note(f"tree attention, trees of 300, room {room}")
    c, m, g = setup([5, 600], heads=1, dim=64, seed=2, room=room)
    run(c, m, inputs(g, 2, 300, 2, 1, 64, torch.bfloat16), [1, 0], mask=tree_mask(g, 2, 300), count=[300, 211], what="trees")


@pytest.mark.parametrize("nodes", [2, 40], ids=["few rows", "many rows"])
@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])
def test_wrong_pages_stand_for_the_first(room, nodes):
    """A table entry out of range is read as page 0, a length past the row's room as that room: the same bits as with
    those numbers in their place."""
    note(f"tree attention, page numbers and a length out of range, {nodes} nodes, room {room}")
    from copy_reduce_amd.torch_api import tree_attention
    c, m, g = setup([100, 40, 9], heads=1, room=room)
    for p in c.pools:
        p.copy_(torch.randn(p.shape, generator=g))
    x = [t.cuda() for t in inputs(g, 3, nodes, 2, 1, 64, torch.bfloat16)]
    wrong = {(0, 2): -5, (0, 3): c.num_pages, (0, 6): -2 ** 31, (1, 1): 2 ** 31 - 1}
    for (q, j), page in wrong.items():
        c.table[q, j] = page
    c.lens[1], c.lens[2] = 1 << 30, -3
    got = tree_attention(*x, c, 0, ints([0, 1, 2]))
    for q, j in wrong:
        c.table[q, j] = 0
    c.lens[1], c.lens[2] = c.max_pages * c.page_tokens, 0
    want = tree_attention(*x, c, 0, ints([0, 1, 2]))
    assert bool(torch.isfinite(want[0]).all()) and bool(torch.isfinite(want[1]).all())
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
