"""GPU tests of attention over a window of the paged cache with sinks (tb_view_attention) against its definition in 64
bits.  The error bounds are those of test_gpu_tree_attention.py: the arithmetic is the same, over fewer keys."""
import math

import pytest
import torch

from gpu_util import note
from serve_model import window_attention
from test_gpu_tree_attention import compare, inputs, ints, setup, tree_mask

pytestmark = pytest.mark.gpu


def depths_of(mask):
    """Depths of the trees whose ancestor masks these are."""
    return sum(((mask >> i) & 1).sum(-1) for i in range(64)).to(torch.int32) - 1


def run(c, m, q, k, v, seqs, window, sinks, mask=None, nodes=None, depths=None, scale=None, what="", **kw):
    from copy_reduce_amd.torch_api import tree_attention
    got = tree_attention(q.cuda(), k.cuda(), v.cuda(), c, 0, ints(seqs), mask=None if mask is None else mask.cuda(),
                         nodes=None if nodes is None else ints(nodes), scale=scale, window=window, sinks=sinks,
                         depths=None if depths is None else depths.cuda(), **kw)
    ref = window_attention(m, 0, q, k, v, seqs, mask, nodes, scale, window, sinks, depths)
    compare(got, ref, max(m.lens) + q.shape[1], q.shape[3], q.dtype, what)
    return got


LENS = [0, 1, 5, 31, 37, 128, 200, 333]


@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (2, 0), (7, 1), (33, 4), (64, 0), (100, 17), (130, 500), (1000, 4), (2 ** 32 - 1, 5)])
@pytest.mark.parametrize("t", [1, 5, 40])
def test_windows(t, window, sinks, room):
    """Every border: windows shorter than the tree, longer than the context, sinks that reach into them or past them."""
    note(f"window {window} sinks {sinks}, chains of {t}, room {room}")
    c, m, g = setup(LENS, heads=2, dim=64, pt=5, seed=t + window % 97, room=max(room, 40))
    q, k, v = inputs(g, len(LENS), t, 4, 2, 64, torch.bfloat16)
    run(c, m, q, k, v, [3, 0, 7, 1, 2, 6, 5, 4], window, sinks, what="chain")


@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("layout,pt", [("token", 16), ("head", 16), ("token", 1), ("head", 20)])
def test_shapes(dim, dtype, layout, pt, room):
    note(f"window attention dim {dim} {dtype} {layout} pages of {pt} room {room}")
    c, m, g = setup([3, 97, 260, 301], heads=2, dim=dim, pt=pt, layout=layout, dtype=dtype, seed=dim + pt, room=room)
    for t, hq in ((1, 2), (3, 8), (13, 14)):   # 1, 12 and 91 rows a head
        q, k, v = inputs(g, 4, t, hq, 2, dim, dtype)
        run(c, m, q, k, v, [2, 0, 3, 1], 50, 6, what=f"{t} nodes")


@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])
@pytest.mark.parametrize("t,group", [(4, 4), (33, 1), (64, 5), (70, 4), (130, 1)])
@pytest.mark.parametrize("window,sinks", [(3, 2), (40, 0), (150, 9)])
def test_trees(t, group, window, sinks, room):
    """Ragged trees: depths that are no node's number, padding nodes, a sequence without nodes and one without a row."""
    note(f"window {window} sinks {sinks}, trees of {t} nodes, {group} rows each, room {room}")
    c, m, g = setup([300, 0, 77, 160], heads=2, dim=64, pt=16, seed=t, room=room)
    q, k, v = inputs(g, 6, t, 2 * group, 2, 64, torch.bfloat16)
    mask = tree_mask(g, 6, t)
    run(c, m, q, k, v, [2, 0, -1, 3, 1, 2], window, sinks, mask, [t, t - 3, t, 0, t, 1], depths_of(mask), what="trees")


def test_depths_out_of_range_are_taken_within():
    note("depths below 0 and past the tree")
    c, m, g = setup([90, 40], heads=1, dim=64, pt=8, dtype=torch.float16)
    q, k, v = inputs(g, 2, 6, 2, 1, 64, torch.float16)
    depths = torch.tensor([[0, -5, 2 ** 31 - 1, 3, -2 ** 31, 9], [0, 1, 2, 3, 4, 5]], dtype=torch.int32)
    run(c, m, q, k, v, [0, 1], 20, 3, nodes=[5, 6], depths=depths)


@pytest.mark.parametrize("t,group", [(5, 2), (5, 16)])
@pytest.mark.parametrize("poison", [math.nan, math.inf, -math.inf])
def test_what_is_not_seen_has_no_effect(t, group, poison):
    """Not finite: all that lies between the sinks and the windows, and what the deeper nodes do not see any more."""
    note(f"{poison} outside the windows, {t} nodes of {group} rows")
    n, window, sinks = 120, 30, 4
    c, m, g = setup([n], heads=1, dim=64, pt=16, seed=5)
    q, k, v = inputs(g, 1, t, group, 1, 64, torch.bfloat16)
    clean = run(c, m, q, k, v, [0], window, sinks)[0].cpu()
    by_token, at = m.by_token(), m.table[0]
    first = n + 1 - window   # the first token that the root sees, and no deeper node
    for j in list(range(sinks, first + 1)):
        by_token[:, at[j // 16], j % 16] = poison
    for i, p in enumerate(c.pools):
        p.copy_(m.kv[i])
    from copy_reduce_amd.torch_api import tree_attention
    out = tree_attention(q.cuda(), k.cuda(), v.cuda(), c, 0, ints([0]), window=window, sinks=sinks)[0].cpu()
    assert torch.equal(out[:, 1:], clean[:, 1:])   # all but the root
    assert bool(out[:, 0].isnan().any()) or not bool(torch.isfinite(out[:, 0]).all())


def test_an_infinite_value_in_the_zone_is_the_root_s():
    note("an infinite value that only the root sees")
    n, window = 70, 20
    c, m, g = setup([n], heads=1, dim=64, pt=16, seed=6)
    q, k, v = inputs(g, 1, 3, 2, 1, 64, torch.bfloat16)
    from copy_reduce_amd.torch_api import tree_attention
    clean = tree_attention(q.cuda(), k.cuda(), v.cuda(), c, 0, ints([0]), window=window)[0].cpu()
    j = n + 1 - window
    m.by_token()[1, m.table[0][j // 16], j % 16, 0, 7] = math.inf
    c.pools[1].copy_(m.kv[1])
    out = tree_attention(q.cuda(), k.cuda(), v.cuda(), c, 0, ints([0]), window=window)[0].cpu()
    assert torch.equal(out[:, 1:], clean[:, 1:])
    assert bool(torch.isinf(out[0, 0, :, 7]).all())
    rest = [e for e in range(64) if e != 7]
    assert torch.equal(out[0, 0][:, rest], clean[0, 0][:, rest])


def test_a_window_past_everything_is_the_whole_context():
    """The two kernels add in another order; both are within the bound of the definition without a window."""
    note("window past the context")
    c, m, g = setup([257, 90], heads=2, dim=128, pt=16, seed=8)
    for t in (1, 30):
        q, k, v = inputs(g, 2, t, 8, 2, 128, torch.bfloat16)
        got = run(c, m, q, k, v, [0, 1], 10 ** 6, 0)
        ref = window_attention(m, 0, q, k, v, [0, 1])
        compare(got, ref, 300, 128, q.dtype, "no window")


def test_long_contexts_by_shares():
    """Windows over long sequences that several workgroups share, and a table wider than the list of a workgroup's pages."""
    note("windows of 5,000 in 9,000 tokens, pages of 1")
    c, m, g = setup([9000, 20, 6000], heads=1, dim=64, pt=1, dtype=torch.float16, seed=9, room=200000)
    for t in (1, 20):
        q, k, v = inputs(g, 3, t, 2, 1, 64, torch.float16)
        run(c, m, q, k, v, [0, 1, 2], 5000, 100, what=f"{t} nodes")


def test_scale_and_strides():
    note("negative scale, strided inputs")
    c, m, g = setup([100, 60], heads=2, dim=64, pt=16, seed=10)
    q, k, v = inputs(g, 2, 4, 4, 2, 64, torch.bfloat16)
    wide = torch.zeros(2, 4, 4, 2, 64, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :, :, 1]
    from copy_reduce_amd.torch_api import tree_attention
    qs = torch.stack([q, q], 3).cuda()[:, :, :, 1]
    got = tree_attention(qs, k.cuda(), v.cuda(), c, 0, ints([0, 1]), scale=-0.3, out=out, window=25, sinks=2)
    compare(got, window_attention(m, 0, q, k, v, [0, 1], scale=-0.3, window=25, sinks=2), 110, 64, q.dtype, "strided")
    assert not bool(wide[:, :, :, 0].any())


@pytest.mark.parametrize("batch,t,group", [(16, 64, 4), (64, 1, 4)], ids=["rows divided", "whole sequences"])
def test_batches_that_fill_the_chip(batch, t, group):
    """So many sequences with windows of 800 that no keys are shared out: many rows are divided instead, few go with a
    workgroup a sequence."""
    note(f"{batch} sequences of {t} nodes, windows of 800")
    lens = [1 + (i * 397) % 1100 for i in range(batch)]
    c, m, g = setup(lens, heads=8, dim=128, pt=32, seed=batch, room=8192)
    q, k, v = inputs(g, batch, t, 8 * group, 8, 128, torch.bfloat16)
    order = torch.randperm(batch, generator=g).tolist()
    if t == 1:
        run(c, m, q, k, v, order, 800, 4, what="single tokens")
    else:
        mask = tree_mask(g, batch, t)
        run(c, m, q, k, v, order, 800, 4, mask, [t - (i % 3) * 20 for i in range(batch)], depths_of(mask), what="trees")


@pytest.mark.parametrize("fp4", [False, True], ids=["16 bits", "4 bits"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_the_same_call_gives_the_same_result(dim, dtype, fp4):
    """Many calls in a row, each form after another one whose values are still in registers and LDS."""
    from copy_reduce_amd.torch_api import PagedCache, fp4_head_bytes, tree_attention
    note(f"the same calls again and again, dim {dim} {dtype} 4 bits: {fp4}")
    c, m, g = setup([3, 97, 260, 301], heads=2, dim=dim, pt=16, layout="token", dtype=dtype, seed=dim, room=0)
    if fp4:
        kv = torch.zeros(2, c.num_pages, 16, 2, fp4_head_bytes(dim), dtype=torch.uint8, device="cuda")
        small = PagedCache(kv, 16, c.max_seqs, c.max_pages, fp4=dtype)
        seqs, lens = ints([0, 1, 2, 3]), ints([3, 97, 260, 301])
        small.resize(seqs, lens)
        who = ints([q for q, n in enumerate([3, 97, 260, 301]) for _ in range(n)])
        at = ints([p for n in [3, 97, 260, 301] for p in range(n)])
        small.append(c.read(who, at), who, at)
        c = small
    s = ints([2, 0, 3, 1])
    for t, hq in ((1, 2), (3, 8), (1, 8), (4, 4)):
        q, k, v = [x.cuda() for x in inputs(g, 4, t, hq, 2, dim, dtype)]
        for window in (50, None, 90):
            got = [tree_attention(q, k, v, c, 0, s, window=window, sinks=6 if window else 0) for _ in range(150)]
            out, lse = torch.stack([o for o, _ in got]), torch.stack([x for _, x in got])
            assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse)), (t, hq, window)
