"""GPU tests of a paged cache held in 4 bits: what append() rounds to, byte for byte against a plain model, what read()
gives back, the calls that move its pages, and attention over it against the definition in 64 bits.

Attention's bounds are those of test_gpu_tree_attention.py: what the cache holds are numbers of the element type, so that the
products are as exact as in 16 bits."""
import math

import pytest
import torch

from cache_model import Model
from gpu_util import note, require_gpu
from serve_model import LIMITS, decode, encode, head_bytes, window_attention
from test_gpu_tree_attention import compare, inputs, ints, tree_mask
from test_gpu_window_attention import depths_of

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16]
IDS = ["bf16", "fp16"]


def make(lens, heads=2, dim=64, pt=16, layout="token", dtype=torch.bfloat16, layers=1, seed=0, pad=0, room=0, spare=3, rows=0):
    """A cache in 4 bits of sequences of these lengths with random contents, its model in numbers, and a generator.
    What no sequence holds is NaN."""
    require_gpu()
    from copy_reduce_amd.torch_api import PagedCache, fp4_head_bytes
    assert fp4_head_bytes(dim) == head_bytes(dim)
    g = torch.Generator().manual_seed(seed)
    seqs, width = max(rows, 1, len(lens)), max(1, max([-(-n // pt) for n in [room, *lens]])) + 1
    pages = sum(-(-n // pt) for n in lens) + spare
    page = (pt, heads) if layout == "token" else (heads, pt)
    m = Model(pages, pt, seqs, width, torch.full((2 * layers, pages) + page + (dim,), math.nan, dtype=dtype), layout)
    m.stack = torch.randperm(pages, generator=g).tolist()
    m.resize(list(range(len(lens))), list(lens))
    hb = head_bytes(dim)
    raw = torch.full((2 * layers, pages) + page + (hb,), 255, dtype=torch.uint8)
    by_token, raw_by_token = m.by_token(), raw if layout == "token" else raw.transpose(2, 3)
    for q, n in enumerate(lens):
        for p in range(n):
            x = encode(torch.randn(2 * layers, heads, dim, generator=g).to(dtype))
            raw_by_token[:, m.table[q][p // pt], p % pt] = x
            by_token[:, m.table[q][p // pt], p % pt] = decode(x, dim).to(dtype)
    stride = pt * heads * hb + pad
    room_ = torch.full((2 * layers, pages * stride), 255, dtype=torch.uint8, device="cuda")
    inner = (hb * heads, hb, 1) if layout == "token" else (hb * pt, hb, 1)
    pools = [r.as_strided((pages,) + page + (hb,), (stride,) + inner) for r in room_]
    for i, p in enumerate(pools):
        p.copy_(raw[i])
    c = PagedCache(pools, pt, seqs, width, layout=layout, fp4=dtype)
    c.state.copy_(torch.from_numpy(m.state(c.state.cpu().numpy())).to(torch.int32))
    return c, m, g


def run(c, m, q, k, v, seqs, mask=None, nodes=None, scale=None, window=None, sinks=0, depths=None, what="", **kw):
    from copy_reduce_amd.torch_api import tree_attention
    got = tree_attention(q.cuda(), k.cuda(), v.cuda(), c, 0, ints(seqs), mask=None if mask is None else mask.cuda(),
                         nodes=None if nodes is None else ints(nodes), scale=scale, window=window, sinks=sinks,
                         depths=None if depths is None else depths.cuda(), **kw)
    ref = window_attention(m, 0, q, k, v, seqs, mask, nodes, scale, window, sinks, depths)
    compare(got, ref, max(m.lens) + q.shape[1], q.shape[3], q.dtype, what)
    return got


def hard_rows(dtype, n, heads, dim, g):
    """Rows whose blocks have magnitudes all over the type's range, ties, zeros of both signs, limits, and values that
    are not finite."""
    x = torch.randn(n, heads, dim, generator=g).double()
    y = x.view(n, heads, dim // 32, 32)
    y *= torch.exp2(torch.randint(-30, 16, y.shape[:3], generator=g).double())[..., None]
    y[0] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4) * 2.0 ** -3   # ties
    y[1] = -y[0]
    y[2] = 0.0
    y[2, ..., 1] = -0.0
    big = torch.finfo(dtype).max
    y[3, ..., 0], y[4, ..., 5], y[5, ..., 31] = big, -big, torch.finfo(dtype).tiny
    y[6] = 0.0
    y[6, ..., 3] = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps   # the smallest subnormal
    for e in range(-6, 6):   # both sides of the border where a block's power changes
        y[7 + (e + 6) % 3, ..., e + 6] = 7 * 2.0 ** (e + LIMITS[dtype][1] - 20)
    x = x.to(dtype)
    z = x.view(n, heads, dim // 32, 32)
    z[11, :, 0, 4], z[12, :, -1, 31], z[13, :, 0, 0] = math.nan, math.inf, -math.inf
    return x


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 256, 512])
@pytest.mark.parametrize("layout,pt,pad", [("token", 16, 0), ("head", 5, 12)])
def test_append_rounds_as_defined(dim, dtype, layout, pt, pad):
    note(f"append in 4 bits: dim {dim} {dtype} {layout}")
    heads = 3
    c, m, g = make([20, 33], heads=heads, dim=dim, pt=pt, layout=layout, dtype=dtype, layers=1, pad=pad)
    before = [p.clone() for p in c.pools]
    new = torch.stack([hard_rows(dtype, 16, heads, dim, g), torch.randn(16, heads, dim, generator=g).to(dtype)])
    seqs, at = [1, 0, 1, -1] * 4, [32, 5, 0, 7, 31, 19, 12, 0, 13, 0, 4, 1, 9, 7, 22, 3]
    index = torch.randperm(16, generator=g).tolist()
    c.append(new.cuda(), ints(seqs), ints(at), ints(index))
    want = encode(new)
    for p in range(2):
        exp = before[p].cpu()
        by = exp if layout == "token" else exp.transpose(1, 2)
        for q, pos, x in zip(seqs, at, index):
            if q >= 0:
                by[m.table[q][pos // pt], pos % pt] = want[p, x]
        assert torch.equal(c.pools[p].cpu(), exp)
    assert c.flags() == 0
    got = c.read(ints(seqs), ints(at)).cpu()
    for i, (q, x) in enumerate(zip(seqs, index)):
        exp = decode(want[:, x], dim) if q >= 0 else torch.zeros(2, heads, dim, dtype=torch.float64)
        assert torch.equal(got[:, i].double().nan_to_num(1e30), exp.nan_to_num(1e30))


@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("dim,heads,n", [(32, 1, 1000), (32, 70, 40), (64, 2, 900), (96, 5, 333), (128, 9, 301), (192, 11, 64),
                                         (512, 1, 129), (2080, 1, 13), (4096, 3, 7)])
def test_lists_of_many_tokens_and_wide_heads(dim, heads, n, layout):
    """More tokens than a workgroup has, in any order with padding between them, and heads that many waves share."""
    note(f"{n} tokens in 4 bits: {heads} heads of {dim} {layout}")
    g = torch.Generator().manual_seed(dim + n)
    lens = [n, n // 3 + 1]
    c, m, _ = make(lens, heads=heads, dim=dim, pt=7, layout=layout, layers=2)
    before = [p.clone() for p in c.pools]
    order = torch.randperm(sum(lens), generator=g).tolist()
    where = [(0, p) if p < n else (1, p - n) for p in order]
    where = [(-1, 5) if i % 10 == 3 else w for i, w in enumerate(where)]
    new = torch.randn(4, len(where) + 5, heads, dim, generator=g).to(torch.bfloat16)
    index = torch.randperm(len(where) + 5, generator=g).tolist()[:len(where)]
    seqs, at = ints([q for q, _ in where]), ints([p for _, p in where])
    c.append(new.cuda(), seqs, at, ints(index))
    want = encode(new)
    for p in range(4):
        exp = before[p].cpu()
        by = exp if layout == "token" else exp.transpose(1, 2)
        for (q, pos), x in zip(where, index):
            if q >= 0:
                by[m.table[q][pos // 7], pos % 7] = want[p, x]
        assert torch.equal(c.pools[p].cpu(), exp)
    assert c.flags() == 0
    got = c.read(seqs, at).cpu()
    exp = decode(want[:, index], dim).to(torch.bfloat16)
    exp[:, [i for i, (q, _) in enumerate(where) if q < 0]] = 0
    assert torch.equal(got, exp)


def test_more_work_than_a_grid_has_room_for():
    """4.4 million listed tokens of 9 heads of 1,024, a workgroup each: all but a few are padding."""
    note("a list of 4.4 million tokens in 4 bits")
    n, real = 4_400_000, [0, 1, 999_999, 2_097_152, 4_194_304, 4_399_999]
    c, m, g = make([len(real)], heads=9, dim=1024, pt=4)
    new = torch.randn(2, 3, 9, 1024, generator=g).to(torch.bfloat16)
    seqs, at, index = [torch.full((n,), x, dtype=torch.int32) for x in (-1, 0, 1)]
    for i, r in enumerate(real):
        seqs[r], at[r], index[r] = 0, i, i % 3
    c.append(new.cuda(), seqs.cuda(), at.cuda(), index.cuda())
    got = c.read(ints([0] * len(real)), ints(list(range(len(real))))).cpu()
    assert c.flags() == 0
    assert torch.equal(got, decode(encode(new), 1024).to(torch.bfloat16)[:, [i % 3 for i in range(len(real))]])


def test_every_value_of_both_types():
    """Each of the 65,536 bit patterns as an element beside a largest one that sets the power."""
    for dtype in DTYPES:
        note(f"every pattern of {dtype}")
        c, m, g = make([16], heads=2, dim=64, pt=16, dtype=dtype, layers=1)
        bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
        bits = bits[torch.isfinite(bits)]
        bits = bits[:len(bits) // 31 * 31].view(-1, 31)
        top = bits.abs().amax(1, keepdim=True)
        blocks = torch.cat([bits, top], 1)
        blocks = torch.cat([blocks, torch.zeros((-len(blocks)) % 64, 32, dtype=dtype)]).view(-1, 16, 2, 64)
        for x in blocks:
            new = torch.stack([x, x])
            c.append(new.cuda(), ints([0] * 16), ints(list(range(16))))
            got = c.read(ints([0] * 16), ints(list(range(16)))).cpu()
            assert torch.equal(got[0].double(), decode(encode(x), 64))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_append_skips_what_it_cannot_do(dtype):
    from copy_reduce_amd import TB_CACHE_RANGE, TB_CACHE_SHARED
    note("4-bit append out of range, into a shared page; read out of range")
    c, m, g = make([20, 0], heads=1, dim=64, pt=8, dtype=dtype, rows=3)
    before = [p.clone() for p in c.pools]
    new = torch.randn(2, 4, 1, 64, generator=g).to(dtype).cuda()
    c.append(new, ints([0, 0, 7, 1]), ints([20, -1, 0, 0]), ints([0, 1, 2, 3]))
    c.append(new, ints([0, 0]), ints([1, 2]), ints([4, -1]))
    assert c.flags(clear=True) == TB_CACHE_RANGE
    got = c.read(ints([0, 0, 9, 0, -1]), ints([20, -1, 0, 3, 3]))
    assert c.flags(clear=True) == TB_CACHE_RANGE
    assert not bool(got[:, [0, 1, 2, 4]].any()) and bool(got[:, 3].any())
    assert all(torch.equal(a, b) for a, b in zip(before, c.pools))
    c.fork(ints([0]), ints([2]))
    c.append(new, ints([0, 2]), ints([3, 19]))
    assert c.flags() == TB_CACHE_SHARED
    assert torch.equal(c.read(ints([2]), ints([19]))[:, 0].cpu().double(), decode(encode(new[:, 1].cpu()), 64))
    assert torch.equal(c.read(ints([0]), ints([3])), c.read(ints([2]), ints([3])))


@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("dim", [64, 128])
def test_forks_copies_and_compactions_keep_the_numbers(dim, layout):
    note(f"fork, resize, copy, compact in 4 bits, dim {dim} {layout}")
    c, m, g = make([37, 21, 9], heads=2, dim=dim, pt=8, layout=layout, layers=2, rows=5, spare=12)
    n = sum((37, 21, 9))
    seqs, at = [0] * 37 + [1] * 21 + [2] * 9, [*range(37), *range(21), *range(9)]
    held = c.read(ints(seqs), ints(at))
    c.fork(ints([0]), ints([3]))
    c.resize(ints([1]), ints([0]))
    c.compact()
    kept = [i for i in range(n) if seqs[i] != 1]
    assert torch.equal(c.read(ints([seqs[i] for i in kept]), ints([at[i] for i in kept])), held[:, kept])
    assert torch.equal(c.read(ints([3] * 37), ints(list(range(37)))), held[:, :37])
    other, _, _ = make([0], heads=2, dim=dim, pt=8, layout=layout, layers=2, spare=4)
    other.resize(ints([0]), ints([8]))
    page = int(c.table[0, 1])
    other.copy_pages(other.table[0, :1].clone(), ints([page]), src=c)
    assert torch.equal(other.read(ints([0] * 8), ints(list(range(8)))), held[:, 8:16])
    assert c.flags() == 0 and other.flags() == 0


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("layout,pt,pad", [("token", 16, 0), ("head", 5, 16), ("token", 3, 8)])
def test_read_of_a_cache_in_16_bits(dtype, layout, pt, pad):
    from test_gpu_tree_attention import setup
    note(f"read in 16 bits {layout} pages of {pt}")
    c, m, g = setup([20, 33], heads=3, dim=96, pt=pt, layout=layout, dtype=dtype, layers=2, pad=pad)
    seqs, at = [1, 0, -1, 1, 1], [32, 19, 0, 0, 33]
    by = m.by_token()
    for layer in (None, 0, 1):
        got = c.read(ints(seqs), ints(at), layer=layer).cpu()
        pools = range(4) if layer is None else (2 * layer, 2 * layer + 1)
        for k, p in enumerate(pools):
            for i, (q, pos) in enumerate(zip(seqs, at)):
                exp = by[p, m.table[q][pos // pt], pos % pt] if q >= 0 and pos < m.lens[q] else torch.zeros(3, 96)
                assert torch.equal(got[k, i], exp.to(dtype))
    room = torch.zeros(2, 7, 3, 96, dtype=dtype, device="cuda")
    out = c.read(ints(seqs), ints(at), layer=1, out=room[:, 1:6])
    assert out.data_ptr() == room[:, 1:6].data_ptr() and torch.equal(out.cpu(), got) and not bool(room[:, [0, 6]].any())
    assert c.flags() == 1 << 1


@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("layout,pt", [("token", 16), ("head", 16), ("token", 1), ("head", 5)])
def test_attention_shapes(dim, dtype, layout, pt, room):
    note(f"attention in 4 bits dim {dim} {dtype} {layout} pages of {pt} room {room}")
    c, m, g = make([1, 37, 128, 200], heads=2, dim=dim, pt=pt, layout=layout, dtype=dtype, seed=dim + pt, pad=4 * (pt == 5), room=room)
    for t, hq in ((1, 2), (4, 6), (13, 14)):   # 1, 12 and 91 rows a head
        q, k, v = inputs(g, 4, t, hq, 2, dim, dtype)
        run(c, m, q, k, v, [2, 0, 3, 1], what=f"{t} nodes")
        run(c, m, q, k, v, [2, 0, 3, 1], window=40, sinks=5, what=f"{t} nodes, window")


@pytest.mark.parametrize("room", [0, 8192], ids=["whole", "shares"])
@pytest.mark.parametrize("t,group,dim", [(4, 4, 64), (33, 1, 128), (64, 5, 128), (70, 2, 96), (40, 4, 256)])
def test_attention_trees(t, group, dim, room):
    note(f"trees of {t} over a cache in 4 bits, {group} rows a node, dim {dim}, room {room}")
    c, m, g = make([300, 0, 77, 160], heads=2, dim=dim, pt=16, seed=t, room=room)
    q, k, v = inputs(g, 6, t, 2 * group, 2, dim, torch.bfloat16)
    mask = tree_mask(g, 6, t)
    seqs, nodes = [2, 0, -1, 3, 1, 2], [t, t - 3, t, 0, t, 1]
    run(c, m, q, k, v, seqs, mask, nodes, what="trees")
    run(c, m, q, k, v, seqs, mask, nodes, window=60, sinks=3, depths=depths_of(mask), what="trees, window")


@pytest.mark.parametrize("group", [2, 16])
def test_not_finite_places(group):
    """A block that is NaN, in a place that only the root sees: the root's alone."""
    note(f"a NaN block in the zone, {group} rows a node")
    n, window = 70, 20
    c, m, g = make([n], heads=1, dim=64, pt=16, seed=6)
    q, k, v = inputs(g, 1, 5, group, 1, 64, torch.bfloat16)
    from copy_reduce_amd.torch_api import tree_attention
    clean = tree_attention(q.cuda(), k.cuda(), v.cuda(), c, 0, ints([0]), window=window)[0].cpu()
    j = n + 1 - window
    c.pools[1][m.table[0][j // 16], j % 16, 0, 33] = 255   # the second block of the values
    out = tree_attention(q.cuda(), k.cuda(), v.cuda(), c, 0, ints([0]), window=window)[0].cpu()
    assert torch.equal(out[:, 1:], clean[:, 1:])
    assert bool(out[0, 0, :, 32:].isnan().all()) and torch.equal(out[0, 0, :, :32], clean[0, 0, :, :32])


def test_long_context():
    note("4 bits: 9,000 tokens in pages of 1, shared by workgroups")
    c, m, g = make([20, 20], heads=1, dim=64, pt=1, seed=9, room=200000, spare=9100)
    n = 9000
    new = torch.randn(2, n, 1, 64, generator=g).to(torch.bfloat16)
    c.resize(ints([0]), ints([n]))
    c.append(new.cuda(), ints([0] * n), ints(list(range(n))))
    held = c.read(ints([0] * n), ints(list(range(n)))).cpu()
    m.resize([0], [n])
    for p in range(n):
        m.by_token()[:, m.table[0][p], 0] = held[:, p]
    for t in (1, 20):
        q, k, v = inputs(g, 2, t, 2, 1, 64, torch.bfloat16)
        run(c, m, q, k, v, [0, 1], what=f"{t} nodes")


@pytest.mark.parametrize("heads,pt", [(1, 1), (3, 1), (1, 5), (3, 7)])
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("pad", [0, 4])
def test_pages_that_are_no_multiple_of_16_bytes(heads, pt, layout, pad):
    """Whole pages and tails are moved by 16 bytes at 4-byte alignment; what lies between pages stays as it was."""
    note(f"pages of {pt * heads * 36} bytes and {pad} between, {layout}")
    c, m, g = make([3 * pt + 2, pt, 2 * pt + 1], heads=heads, dim=64, pt=pt, layout=layout, layers=2, rows=6, spare=20, pad=pad)
    lens = [3 * pt + 2, pt, 2 * pt + 1]
    seqs, at = [q for q, n in enumerate(lens) for _ in range(n)], [p for n in lens for p in range(n)]
    held = c.read(ints(seqs), ints(at))
    c.fork(ints([0, 2, 0]), ints([3, 4, 5]))
    for child, parent in ((3, 0), (4, 2), (5, 0)):
        own = [i for i, q in enumerate(seqs) if q == parent]
        assert torch.equal(c.read(ints([child] * lens[parent]), ints(list(range(lens[parent])))), held[:, own])
    c.resize(ints([0, 3]), ints([0, 0]))
    c.compact()
    kept = [i for i, q in enumerate(seqs) if q != 0]
    assert torch.equal(c.read(ints([seqs[i] for i in kept]), ints([at[i] for i in kept])), held[:, kept])
    assert torch.equal(c.read(ints([5] * lens[0]), ints(list(range(lens[0])))), held[:, :lens[0]])
    last = int(c.free_list[0])
    c.copy_pages(ints([last]), c.table[1, :1].clone())
    assert all(torch.equal(p[last], p[int(c.table[1, 0])]) for p in c.pools) and c.flags() == 0
    if pad:
        between = torch.as_strided(c.pools[0], (c.num_pages, pad), (c.pools[0].stride(0), 1), c.pools[0].storage_offset() + pt * heads * 36)
        assert bool((between == 255).all())


def test_pages_past_4_gib():
    """Pages 1.2 GiB apart: places, and what append, read, fork and attention make of them, past 32 bits of bytes."""
    note("4 bits: pools of 6 GiB, pages 1.2 GiB apart")
    require_gpu()
    from copy_reduce_amd.torch_api import PagedCache, fp4_head_bytes
    g = torch.Generator().manual_seed(3)
    pages, pt, heads, dim, apart = 5, 16, 2, 64, (1 << 30) + (200 << 20) + 4
    hb = fp4_head_bytes(dim)
    room = [torch.empty((pages - 1) * apart + pt * heads * hb, dtype=torch.uint8, device="cuda") for _ in range(2)]
    pools = [r.as_strided((pages, pt, heads, hb), (apart, heads * hb, hb, 1)) for r in room]
    c = PagedCache(pools, pt, 3, 5, fp4=torch.bfloat16)
    m = Model(pages, pt, 3, 5, torch.zeros(2, pages, pt, heads, dim, dtype=torch.bfloat16), "token")
    m.stack = list(range(pages - 1, -1, -1))
    n = 50
    c.resize(ints([1]), ints([n]))
    m.resize([1], [n])
    new = torch.randn(2, n, heads, dim, generator=g).to(torch.bfloat16)
    c.append(new.cuda(), ints([1] * n), ints(list(range(n))))
    want = decode(encode(new), dim).to(torch.bfloat16)
    assert torch.equal(c.read(ints([1] * n), ints(list(range(n)))).cpu(), want)
    for p in range(n):
        m.by_token()[:, m.table[1][p // pt], p % pt] = want[:, p]
    for t, hq in ((1, 4), (20, 4)):
        q, k, v = inputs(g, 1, t, hq, heads, dim, torch.bfloat16)
        run(c, m, q, k, v, [1], what=f"{t} nodes")
        run(c, m, q, k, v, [1], window=18, sinks=3, what=f"{t} nodes, window")
    c.fork(ints([1]), ints([0]))
    assert torch.equal(c.read(ints([0] * n), ints(list(range(n)))).cpu(), want) and c.flags() == 0
