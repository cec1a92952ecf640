"""GPU tests of tb_tree_attention against its definition in 64 bits.

Error bounds, derived from the arithmetic that the header promises (u the half
step of the element type, 2^-8 or 2^-11; e = 2^-24 that of fp32):
  scores    a sum of D exact products in fp32: |ds| <= 2 D e S, S = sum |q||k| scale;
            scaling and the change of base of the exponential add 8 e |s| <= 8 e S;
            the exponential itself 4 e relative: each weight is off by the factor
            1 + w, |w| <= (2 D + 8) e S + 8 e, numerator and denominator alike
  weights   rounded to the element type for the second product: a factor 1 + u, and for
            fp16 an absolute 2^-25 each where they are subnormal, against a sum of
            at least 1 (the largest weight)
  sums      n terms in fp32, in any order, split and joined: (n + 64) e relative, twice
  out       |o| u
so |do| <= |o| u + A (u + 2 w + 2 (n + 64) e) + [fp16] n 2^-25 V + 2^-25 (a subnormal result),
A = sum w |v|, V the largest |v|, and |dlse| <= w + (n + 64) e + 4 e |lse|."""
import math

import pytest
import torch

from cache_model import Model, attention
from gpu_util import note, require_gpu

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def setup(lens, heads=2, dim=64, pt=16, layout="token", dtype=torch.bfloat16, layers=1, seed=0, pad=0, spread=1.0, room=0):
    """A cache of sequences of these lengths, pages in a random order, and its model.
    What no sequence holds is NaN.  room: tokens that a row of the table has place for, if more than these; past some
    thousands the keys are cut into shares, below a workgroup takes a whole sequence."""
    require_gpu()
    from copy_reduce_amd.torch_api import PagedCache
    g = torch.Generator().manual_seed(seed)
    seqs, width = max(1, len(lens)), max(1, max([-(-n // pt) for n in [room, *lens]])) + 1
    pages = sum(-(-n // pt) for n in lens) + 3
    page = (pt, heads, dim) if layout == "token" else (heads, pt, dim)
    kv = torch.full((2 * layers, pages) + page, math.nan, dtype=dtype)
    m = Model(pages, pt, seqs, width, kv, layout)
    m.stack = torch.randperm(pages, generator=g).tolist()
    m.resize(list(range(len(lens))), list(lens))
    by_token = m.by_token()
    for q, n in enumerate(lens):
        for p in range(n):
            by_token[:, m.table[q][p // pt], p % pt] = (spread * torch.randn(2 * layers, heads, dim, generator=g)).to(dtype)
    room = torch.full((2 * layers, pages * (pt * heads * dim + pad)), math.nan, dtype=dtype, device="cuda")
    inner = (dim * heads, dim, 1) if layout == "token" else (dim * pt, dim, 1)
    pools = [r.as_strided((pages,) + page, (pt * heads * dim + pad,) + inner) for r in room]
    for i, p in enumerate(pools):
        p.copy_(m.kv[i])
    c = PagedCache(pools, pt, seqs, width, layout=layout)
    c.state.copy_(torch.from_numpy(m.state(c.state.cpu().numpy())).to(torch.int32))
    return c, m, g


def inputs(g, b, t, hq, hk, d, dtype, spread=1.0):
    return [(spread * torch.randn(b, t, h, d, generator=g)).to(dtype) for h in (hq, hk, hk)]


def tree_mask(g, b, t):
    """Ancestor masks of random trees, node 0 the root: (words, parents)."""
    words = torch.zeros(b, t, (t + 63) // 64, dtype=torch.int64)
    for i in range(b):
        for x in range(t):
            sees = {x}
            if x:
                p = int(torch.randint(0, x, (1,), generator=g))
                sees |= {u for u in range(t) if int(words[i, p, u // 64]) >> (u % 64) & 1}
            for u in sees:
                bit = 1 << (u % 64)
                words[i, x, u // 64] |= bit - (1 << 64) if bit >> 63 else bit
    return words


def bounds(ref, n, d, dtype):
    out, lse, a, s, big = ref
    u = torch.finfo(dtype).eps / 2
    w = (2 * d + 8) * E * s + 8 * E
    tol = out.abs() * u + a * (u + 2 * w + 2 * (n + 64) * E)[..., None] + 1e-30
    if dtype == torch.float16:
        tol = tol + (n * 2.0 ** -25 * big)[..., None] + 2.0 ** -25
    return tol, w + (n + 64) * E + 4 * E * lse.abs().nan_to_num(0, 0, 0)


def compare(got, ref, n, d, dtype, what):
    out, lse = got[0].double().cpu(), got[1].double().cpu()
    tol_o, tol_l = bounds(ref, n, d, dtype)
    empty = torch.isneginf(ref[1])
    assert torch.equal(torch.isneginf(lse), empty), f"{what}: rows that see nothing"
    assert not out[empty].any(), f"{what}: a row that sees nothing is not 0"
    dl = ((lse - ref[1]).abs() / tol_l)[~empty]
    do = (out - ref[0]).abs() / tol_o
    assert bool(torch.isfinite(out).all())
    assert dl.numel() == 0 or float(dl.max()) <= 1, f"{what}: lse off by {float(dl.max()):.3g} of the bound"
    assert do.numel() == 0 or float(do.max()) <= 1, f"{what}: out off by {float(do.max()):.3g} of the bound"


def run(c, m, q, k, v, seqs, mask=None, nodes=None, scale=None, what="", **kw):
    from copy_reduce_amd.torch_api import tree_attention
    got = tree_attention(q.cuda() if not q.is_cuda else q, k.cuda() if not k.is_cuda else k, v.cuda() if not v.is_cuda else v, c, 0,
                         ints(seqs), mask=None if mask is None else mask.cuda(), nodes=None if nodes is None else ints(nodes), scale=scale, **kw)
    ref = attention(m, 0, q.cpu(), k.cpu(), v.cpu(), seqs, mask, nodes, scale)
    compare(got, ref, max(m.lens) + q.shape[1], q.shape[3], q.dtype, what)
    return got


@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("layout,pt", [("token", 16), ("head", 16), ("token", 1), ("head", 5), ("token", 20), ("token", 64), ("head", 96)])
def test_shapes(dim, dtype, layout, pt, room):
    note(f"tree attention dim {dim} {dtype} {layout} pages of {pt}")
    c, m, g = setup([1, 37, 128, 200], heads=2, dim=dim, pt=pt, layout=layout, dtype=dtype, seed=dim + pt, pad=8 * (pt == 5), room=room)
    q, k, v = inputs(g, 4, 5, 6, 2, dim, dtype)
    run(c, m, q, k, v, [2, 0, 3, 1], what="chain")


@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])
@pytest.mark.parametrize("nodes", [1, 2, 3, 7, 8, 15, 16, 17, 31, 33, 63, 64, 65, 100, 130])
@pytest.mark.parametrize("group", [1, 4, 7])
def test_nodes_and_groups(nodes, group, room):
    note(f"tree attention {nodes} nodes, {group} query heads a key head")
    c, m, g = setup([70, 0, 259], heads=1, seed=nodes, room=room)
    q, k, v = inputs(g, 3, nodes, group, 1, 64, torch.bfloat16)
    run(c, m, q, k, v, [0, 1, 2], mask=tree_mask(g, 3, nodes), nodes=[nodes, nodes, nodes - nodes // 3], what="tree")


@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])
@pytest.mark.parametrize("lens", [[0], [1], [15], [16], [31], [32], [33], [127], [128], [129], [255, 256, 257], [511, 513, 1], [1025, 0, 3], [4097],
                                  [2000] + [1] * 30])
@pytest.mark.parametrize("nodes", [1, 6])
def test_lengths(lens, nodes, room):
    note(f"tree attention lengths {lens[:4]} {nodes} nodes")
    c, m, g = setup(lens, heads=2, seed=sum(lens), room=room)
    q, k, v = inputs(g, len(lens), nodes, 8, 2, 64, torch.bfloat16)
    run(c, m, q, k, v, list(range(len(lens))), what="chain")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_long(dtype):
    note(f"tree attention over 20000 tokens {dtype}")
    c, m, g = setup([20000, 3], heads=1, dim=128, dtype=dtype, pt=32)
    q, k, v = inputs(g, 2, 2, 4, 1, 128, dtype)
    run(c, m, q, k, v, [0, 1], what="long")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("dim,pt,layout", [(64, 16, "token"), (96, 20, "head"), (128, 7, "token"), (256, 16, "head"), (128, 128, "head")])
@pytest.mark.parametrize("nodes,group", [(1, 16), (5, 4), (17, 4), (40, 8)])
def test_trees_over_several_shares(dim, pt, layout, dtype, nodes, group):
    """Contexts that several workgroups divide, each part ending anywhere in a page."""
    note(f"tree attention, {nodes} nodes of {group} rows over shares, dim {dim} pages of {pt} {dtype}")
    c, m, g = setup([3000, 0, 1501, 7], heads=2, dim=dim, pt=pt, layout=layout, dtype=dtype, seed=nodes + dim, room=8192)
    q, k, v = inputs(g, 4, nodes, 2 * group, 2, dim, dtype)
    run(c, m, q, k, v, [0, 1, 2, 3], mask=tree_mask(g, 4, nodes), nodes=[nodes, 1, nodes - nodes // 3, nodes], what="shares")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_many_rows_that_are_joined(dim, dtype):
    """16,384 rows and more, some of one share and some of several."""
    note(f"tree attention, many rows over shares, dim {dim} {dtype}")
    c, m, g = setup([2000, 0, 700, 7, 130], heads=2, dim=dim, pt=16, dtype=dtype, seed=dim, room=8192)
    q, k, v = inputs(g, 6, 131, 26, 2, dim, dtype)
    run(c, m, q, k, v, [0, 1, -1, 2, 3, 4], mask=tree_mask(g, 6, 131), nodes=[131, 90, 131, 131, 0, 64], what="many rows")


@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])
@pytest.mark.parametrize("batch,nodes", [(1, 1), (65, 1), (300, 1), (2, 20), (513, 17)])
def test_batches(batch, nodes, room):
    note(f"tree attention batch {batch} {nodes} nodes")
    lens = [(37 * i) % 90 for i in range(batch)]
    c, m, g = setup(lens, heads=1, seed=batch, room=room)
    q, k, v = inputs(g, batch, nodes, 2, 1, 64, torch.bfloat16)
    run(c, m, q, k, v, torch.randperm(batch, generator=g).tolist(), what="batch")


@pytest.mark.parametrize("lens,room,heads,dim,nodes,group", [([4700], 8192, 128, 256, 1, 1), ([4000, 2300, 2049, 5], 0, 64, 64, 17, 1), ([9000], 0, 16, 64, 64, 16)],
                         ids=["few rows", "many rows, whole", "many rows, shares"])
def test_more_pages_than_a_workgroup_keeps(lens, room, heads, dim, nodes, group):
    """Pages of one token: parts of more pages than the 2,048 whose numbers a workgroup keeps."""
    note(f"tree attention, {lens} pages of one token")
    c, m, g = setup(lens, heads=heads, dim=dim, pt=1, room=room)
    q, k, v = inputs(g, len(lens), nodes, heads * group, heads, dim, torch.bfloat16)
    run(c, m, q, k, v, list(range(len(lens))), what="pages of one token")


@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])
def test_masks_that_leave_nothing(room):
    """Rows that see no node, with and without a context; a node that sees all others; none at all."""
    note("tree attention, empty rows")
    c, m, g = setup([0, 40, 0, 0], heads=2, room=room)
    q, k, v = inputs(g, 4, 6, 4, 2, 64, torch.bfloat16)
    mask = torch.zeros(4, 6, 1, dtype=torch.int64)
    mask[0, 2, 0] = 0b111111
    mask[0, 5, 0] = -1            # bits past the last node count for nothing
    mask[2, 0, 0] = 1
    run(c, m, q, k, v, [0, 1, 2, 3], mask=mask, what="masks")
    run(c, m, q, k, v, [0, 1, 2, 3], mask=mask, nodes=[6, 0, 1, 6], what="masks and sizes")
@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])


def test_rows_that_are_not_there(room):
    note("tree attention, padded batch")
    c, m, g = setup([33, 20], heads=2, room=room)
    q, k, v = inputs(g, 5, 3, 4, 2, 64, torch.bfloat16)
    run(c, m, q, k, v, [1, -1, 0, 2, -7], nodes=[3, 3, 2, 3, 9], what="padding")


@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf, 3e38])
def test_masked_values_have_no_effect(value, room):
    """What a row does not see may hold anything: nodes of other branches and padded nodes (the cache's unused tokens are NaN in every test)."""
    note(f"tree attention, {value} in masked places")
    c, m, g = setup([40, 0], heads=2, room=room)
    q, k, v = inputs(g, 2, 40, 4, 2, 64, torch.bfloat16)
    mask = tree_mask(g, 2, 40)
    from copy_reduce_amd.torch_api import tree_attention
    args = dict(mask=mask.cuda(), nodes=ints([37, 40]))
    want = tree_attention(q.cuda(), k.cuda(), v.cuda(), c, 0, ints([0, 1]), **args)
    blind = []                # rows that do not see the changed nodes
    for i, bad in ((0, 5), (0, 20), (1, 3)):
        k[i, bad], v[i, bad] = value, value
        blind.append((i, bad))
    k[0, 37:], v[0, 37:] = value, value
    got = tree_attention(q.cuda(), k.cuda(), v.cuda(), c, 0, ints([0, 1]), **args)
    kept = 0
    for i in range(2):
        for x in range(40):
            if not any(i == j and int(mask[i, x, 0]) >> bad & 1 for j, bad in blind):
                kept += 1
                assert torch.equal(got[0][i, x], want[0][i, x]) and torch.equal(got[1][i, x], want[1][i, x]), (i, x)
    assert kept > 40


def test_seen_values_that_are_not_finite():
    """An infinite value that is seen makes its element infinite, one of each sign NaN; other elements stay."""
    note("tree attention, infinities that are seen")
    from copy_reduce_amd.torch_api import tree_attention
    c, m, g = setup([40], heads=1)
    q, k, v = inputs(g, 1, 3, 1, 1, 64, torch.bfloat16)
    want, _ = tree_attention(q.cuda(), k.cuda(), v.cuda(), c, 0, ints([0]))
    v[0, 0, 0, 7], v[0, 1, 0, 7], v[0, 1, 0, 9] = math.inf, -math.inf, math.nan
    got, _ = tree_attention(q.cuda(), k.cuda(), v.cuda(), c, 0, ints([0]))
    assert float(got[0, 0, 0, 7]) == math.inf and torch.isnan(got[0, 1:, 0, 7]).all() and torch.isnan(got[0, 1:, 0, 9]).all()
    rest = [d for d in range(64) if d not in (7, 9)]
    assert torch.equal(got[..., rest], want[..., rest]) and torch.equal(got[0, 0, 0, 9], want[0, 0, 0, 9])


@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])
@pytest.mark.parametrize("spread", [8.0, 30.0])
def test_sharp_scores(spread, room):
    """Scores of hundreds: single keys decide, running maxima move."""
    note(f"tree attention, scores spread by {spread}")
    c, m, g = setup([700, 64], heads=1, spread=spread ** 0.5, room=room)
    q, k, v = inputs(g, 2, 9, 4, 1, 64, torch.bfloat16, spread ** 0.5)
    run(c, m, q, k, v, [0, 1], mask=tree_mask(g, 2, 9), scale=1.0, what="sharp")
@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])


def test_scale_zero_and_negative(room):
    note("tree attention, scale 0 and negative")
    c, m, g = setup([100], heads=1, room=room)
    q, k, v = inputs(g, 1, 2, 2, 1, 64, torch.bfloat16)
    run(c, m, q, k, v, [0], scale=0.0, what="0")
    run(c, m, q, k, v, [0], scale=-0.3, what="negative")
@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])


def test_strides(room):
    """q, k, v as parts of one projection, out and its rows in a larger tensor; guards stay."""
    note("tree attention, strides")
    c, m, g = setup([90, 33], heads=2, dim=64, room=room)
    fused = torch.randn(2, 4, 8 + 2 + 2, 64, generator=g).to(torch.bfloat16).cuda()
    q, k, v = fused[:, :, :8], fused[:, :, 8:10], fused[:, :, 10:]
    big = torch.full((2, 6, 8, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    run(c, m, q, k, v, [0, 1], out=big[:, 1:5, :, :64], what="strides")
    big[:, 1:5, :, :64] = 7.0
    assert bool((big == 7.0).all())
    by_head = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v)]
    run(c, m, *by_head, [0, 1], what="head-major inputs")
    one = [x[:, :1] for x in (q, k, v)]
    run(c, m, *one, [0, 1], what="one node of a larger tensor")


def test_nothing_to_do():
    note("tree attention, no batch, no nodes")
    from copy_reduce_amd.torch_api import tree_attention
    c, m, g = setup([5], heads=2)
    for b, t in ((0, 3), (1, 0)):
        q, k, v = [x.cuda() for x in inputs(g, b, t, 4, 2, 64, torch.bfloat16)]
        out, lse = tree_attention(q, k, v, c, 0, ints([0] * b))
        assert out.shape == q.shape and lse.shape == (b, t, 4)


def test_same_workspace_again_and_determinism():
    note("tree attention, one workspace for calls in a row")
    from copy_reduce_amd.torch_api import tree_attention, tree_attention_workspace
    c, m, g = setup([3000, 5, 900], heads=2)
    q, k, v = [x.cuda() for x in inputs(g, 3, 4, 8, 2, 64, torch.bfloat16)]
    w = tree_attention_workspace(q, c)
    w.fill_(0xFF)
    first = tree_attention(q, k, v, c, 0, ints([0, 1, 2]), workspace=w)
    other = tree_attention(q, k, v, c, 0, ints([2, 2, 1]), workspace=w)
    again = tree_attention(q, k, v, c, 0, ints([0, 1, 2]), workspace=w)
    free = tree_attention(q, k, v, c, 0, ints([0, 1, 2]))
    for x in (again, free):
        assert torch.equal(first[0], x[0]) and torch.equal(first[1], x[1])
    ref = attention(m, 0, q.cpu(), k.cpu(), v.cpu(), [2, 2, 1])
    compare(other, ref, 3004, 64, torch.bfloat16, "rows twice")
@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])


def test_captured(room):
    """A graph of two calls that share a workspace, replayed over changing lengths and inputs."""
    note("tree attention, captured")
    from copy_reduce_amd.torch_api import tree_attention, tree_attention_workspace
    c, m, g = setup([500, 60], heads=2, room=room)
    q, k, v = [x.cuda() for x in inputs(g, 2, 3, 4, 2, 64, torch.bfloat16)]
    seqs = ints([0, 1])
    w = tree_attention_workspace(q, c)
    tree_attention(q, k, v, c, 0, seqs, workspace=w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = tree_attention(q, k, v, c, 0, seqs, workspace=w)
        b = tree_attention(q, k, v, c, 0, seqs)
    for step, lens in enumerate(([500, 60], [499, 0], [1, 61], [500, 60])):
        m.lens[:] = [min(lens[0], 500), min(lens[1], 60)]
        c.lens.copy_(ints(m.lens))
        q.copy_(torch.randn(q.shape, generator=g).to(q.dtype))
        graph.replay()
        e = tree_attention(q, k, v, c, 0, seqs, workspace=w)
        torch.cuda.synchronize()
        for x in (a, b):
            assert torch.equal(x[0], e[0]) and torch.equal(x[1], e[1]), step
        compare(e, attention(m, 0, q.cpu(), k.cpu(), v.cpu(), [0, 1]), 503, 64, torch.bfloat16, f"step {step}")


def test_two_streams():
    note("tree attention, two calls at once")
    from copy_reduce_amd.torch_api import tree_attention
    c, m, g = setup([5000, 4000], heads=2)
    sets = [[x.cuda() for x in inputs(g, 2, 3, 4, 2, 64, torch.bfloat16)] for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    seqs = ints([0, 1])
    torch.cuda.synchronize()
    got = [tree_attention(*x, c, 0, seqs, stream=s) for x, s in zip(sets, streams)]
    torch.cuda.synchronize()
    for x, y in zip(sets, got):
        compare(y, attention(m, 0, *[z.cpu() for z in x], [0, 1]), 5003, 64, torch.bfloat16, "stream")


def test_second_layer_and_far_pages():
    """Pools past 4 GiB and the second layer's keys and values."""
    note("tree attention, far pages")
    from copy_reduce_amd.torch_api import PagedCache, tree_attention
    pages, pt, d = 70000, 16, 128
    kv = torch.zeros(4, pages, pt, 16, d, dtype=torch.bfloat16, device="cuda")     # 4.3 GiB a pool
    c = PagedCache(kv, pt, 1, 4)
    c.free_list[:pages] = torch.arange(pages, dtype=torch.int32, device="cuda")
    c.resize(ints([0]), ints([50]))
    g = torch.Generator().manual_seed(1)
    new = torch.randn(4, 50, 16, d, generator=g).to(torch.bfloat16)
    c.append(new.cuda(), ints([0] * 50), ints(list(range(50))))
    q, k, v = inputs(g, 1, 2, 16, 16, d, torch.bfloat16)
    got = tree_attention(q.cuda(), k.cuda(), v.cuda(), c, 1, ints([0]))
    m = Model(4, 50, 1, 1, new[:, None].expand(4, 4, 50, 16, d), "token")
    m.resize([0], [50])
    compare(got, attention(m, 1, q, k, v, [0]), 52, d, torch.bfloat16, "far")
@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])


def test_wrong_pages_are_not_followed(room):
    """Table entries out of range give some values, and no access outside the pools."""
    note("tree attention, page numbers out of range")
    from copy_reduce_amd.torch_api import tree_attention
    c, m, g = setup([100, 40], heads=1, room=room)
    c.table[0, 2], c.table[0, 3], c.lens[1] = -5, c.num_pages, 1 << 30
    q, k, v = [x.cuda() for x in inputs(g, 2, 2, 2, 1, 64, torch.bfloat16)]
    tree_attention(q, k, v, c, 0, ints([0, 1]))
    torch.cuda.synchronize()
@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])


def test_serving_run(room):
    """Prompts in, a tree scored, its best path accepted, a fork, a compaction, and the next step over the moved pages."""
    note("tree attention, a serving run")
    from copy_reduce_amd.torch_api import tree_attention
    c, m, g = setup([45, 17, 0, 0], heads=2, dim=128, layers=2, layout="head", room=room)
    for step in range(3):
        t = 5
        q, k, v = inputs(g, 2, t, 4, 2, 128, torch.bfloat16)
        mask = tree_mask(g, 2, t)
        run(c, m, q, k, v, [0, 1], mask=mask, what=f"step {step}")
        path = [[0, 2], [0, 1, 4]]
        new = torch.randn(4, 2 * t, 2, 128, generator=g).to(torch.bfloat16)
        grown = [m.lens[i] + len(path[i]) for i in range(2)]
        args = [i for i in range(2) for _ in path[i]], [m.lens[i] + n for i in range(2) for n in range(len(path[i]))], \
            [i * t + u for i in range(2) for u in path[i]]
        c.resize(ints([0, 1]), ints(grown)), m.resize([0, 1], grown)
        c.append(new.cuda(), *[ints(a) for a in args]), m.append(new, *args)
        if step == 0:
            c.fork(ints([1]), ints([2])), m.fork([1], [2])
            c.resize(ints([0]), ints([20])), m.resize([0], [20])
        c.compact(), m.compact()
        m.check(c, f"step {step}")
        assert c.flags() == 0
    run(c, m, *inputs(g, 3, 1, 4, 2, 128, torch.bfloat16), [2, 0, 1], what="single tokens at the end")


def test_refusals():
    note("tree attention, refusals")
    from copy_reduce_amd import TBError
    from copy_reduce_amd.torch_api import tree_attention
    c, m, g = setup([10], heads=2)
    q, k, v = [x.cuda() for x in inputs(g, 1, 2, 4, 2, 64, torch.bfloat16)]
    seqs = ints([0])
    for bad in (dict(q=q.half()), dict(q=q[..., :32]), dict(k=k[:, :1]), dict(v=v.float()), dict(layer=1), dict(seqs=seqs.long()),
                dict(mask=torch.zeros(1, 2, 2, dtype=torch.int64, device="cuda")), dict(mask=torch.zeros(1, 2, 1, dtype=torch.int64)),
                dict(nodes=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(out=torch.zeros(1, 2, 4, 64, device="cuda")),
                dict(lse=torch.zeros(1, 2, 4, dtype=torch.float64, device="cuda")), dict(q=q.transpose(2, 3)), dict(k=k.cpu())):
        a = dict(q=q, k=k, v=v, cache=c, layer=0, seqs=seqs)
        a.update(bad)
        with pytest.raises(ValueError):
            tree_attention(**a)
    with pytest.raises(TBError):      # a head of 72 elements starts off a 16-byte boundary
        room = torch.zeros(1, 2, 4, 68, dtype=torch.bfloat16, device="cuda")
        tree_attention(room[..., :64], k, v, c, 0, seqs)
    with pytest.raises(TBError):
        tree_attention(q, k, v, c, 0, seqs, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TBError):      # three query heads over two key heads
        tree_attention(q[:, :, :3], k, v, c, 0, seqs)


def test_inputs_that_want_a_gradient_are_refused():
    note("tree attention, gradients")
    from copy_reduce_amd.torch_api import tree_attention
    c, m, g = setup([10], heads=2)
    q, k, v = [x.cuda() for x in inputs(g, 1, 2, 4, 2, 64, torch.bfloat16)]
    want = tree_attention(q, k, v, c, 0, ints([0]))
    for x in (q, k, v):
        x.requires_grad_()
        with pytest.raises(ValueError):
            tree_attention(q, k, v, c, 0, ints([0]))
        with torch.no_grad():
            got = tree_attention(q, k, v, c, 0, ints([0]))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        x.requires_grad_(False)


@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])
def test_two_graphs_share_a_workspace(room):
    """Captured apart, of other batches and trees, replayed in turn over growing lengths with eager calls between."""
    note("tree attention, two graphs with one workspace")
    from copy_reduce_amd.torch_api import tree_attention, tree_attention_workspace
    c, m, g = setup([600, 300, 90], heads=2, room=room)
    small = [x.cuda() for x in inputs(g, 2, 1, 4, 2, 64, torch.bfloat16)]
    large = [x.cuda() for x in inputs(g, 3, 9, 8, 2, 64, torch.bfloat16)]
    w = max((tree_attention_workspace(x[0], c) for x in (small, large)), key=lambda t: t.nbytes)
    calls = [(small, ints([2, 0])), (large, ints([0, 1, 2]))]
    graphs, outs = [], []
    for x, seqs in calls:
        tree_attention(*x, c, 0, seqs, workspace=w)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(tree_attention(*x, c, 0, seqs, workspace=w))
        graphs.append(graph)
    for lens in ([1, 0, 90], [600, 300, 90], [257, 128, 31], [600, 1, 0]):
        c.lens.copy_(ints(lens))
        for graph in graphs:
            graph.replay()
        got = [(o.clone(), l.clone()) for o, l in outs]
        for (x, seqs), (o, l) in zip(calls, got):
            eo, el = tree_attention(*x, c, 0, seqs, workspace=w)
            torch.cuda.synchronize()
            assert torch.equal(o, eo) and torch.equal(l, el), lens
        m.lens[:] = lens
        compare(got[1], attention(m, 0, *[x.cpu() for x in large], [0, 1, 2]), 609, 64, torch.bfloat16, f"lengths {lens}")
