"""GPU tests of the paged cache: every call against the plain model of
cache_model.py, bookkeeping and bytes equal."""
import random

import pytest
import torch

from cache_model import Model
from copy_reduce_amd import TB_CACHE_SHARED
from gpu_util import note, require_gpu

pytestmark = pytest.mark.gpu


def make(pages=23, pt=4, seqs=9, width=7, heads=2, dim=8, layers=1, layout="token", dtype=torch.bfloat16, pad=0, shift=0):
    """A cache and its model, pools filled; pad: elements between pages, shift: elements the pools start off
    a 16-byte boundary."""
    require_gpu()
    from copy_reduce_amd.torch_api import PagedCache
    page = (pt, heads, dim) if layout == "token" else (heads, pt, dim)
    n, size = 2 * layers, pt * heads * dim
    g = torch.Generator().manual_seed(pages * 131 + pt)
    kv = torch.randint(0, 256, (n, pages) + page + (torch.empty(0, dtype=dtype).element_size(),), generator=g,
                       dtype=torch.uint8).view(dtype).view((n, pages) + page)
    pools = []
    for i in range(n):
        room = torch.zeros(shift + pages * (size + pad), dtype=dtype, device="cuda")
        strides = (dim * heads, dim, 1) if layout == "token" else (dim * pt, dim, 1)
        pool = room.as_strided((pages,) + page, (size + pad,) + strides, shift)
        pool.copy_(kv[i])
        pools.append(pool)
    return PagedCache(pools, pt, seqs, width, layout=layout), Model(pages, pt, seqs, width, kv, layout)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rows(cache, n, seed=1):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(len(cache.pools), n, cache.heads, cache.head_dim, generator=g).to(cache.dtype)


SHAPES = [dict(), dict(layout="head"), dict(pt=1, width=20), dict(pt=5, heads=3, dim=6), dict(dim=3, layout="head"),
          dict(pad=8), dict(pad=3), dict(shift=1), dict(shift=8, pad=8, layout="head"), dict(layers=3, dtype=torch.float16),
          dict(pt=16, heads=4, dim=128, width=3), dict(pt=64, heads=8, dim=128, width=2, layout="head"),
          dict(heads=1, dim=1056, dtype=torch.float16), dict(dtype=torch.float32), dict(dtype=torch.uint8, dim=5)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_all_calls_in_a_row(shape):
    """A serving run: prompts come, are forked, appended to, freed, compacted."""
    note(f"paged cache, calls in a row, {shape}")
    c, m = make(**shape)
    cap = m.MP * m.pt
    m.check(c, "new")

    def both(name, *args):
        getattr(c, name)(*[ints(a) if isinstance(a, list) else a.cuda() if isinstance(a, torch.Tensor) else a for a in args])
        getattr(m, name)(*args)
        m.check(c, f"{name} {args if not isinstance(args[0] if args else 0, torch.Tensor) else args[1:]}")

    first = min(2 * m.pt + m.pt // 2, cap)
    both("resize", [3, 0, 5], [first, m.pt, 1])
    pos = list(range(first)) + list(range(m.pt)) + [0]
    both("append", rows(c, len(pos) + 2), [3] * first + [0] * m.pt + [5], pos, [(7 * i + 1) % (len(pos) + 2) for i in range(len(pos))])
    both("fork", [3, 3, -1, 0, 5], [1, 8, 2, 7, 4])
    both("resize", [1, 8], [min(first + 1, cap), min(first + m.pt, cap)])
    both("append", rows(c, 2, 5), [1, 8], [first - 1 if first == cap else first, first - 1])
    both("resize", [3, 0, -4, 7], [0, 0, 5, 1])
    both("compact")
    both("compact")
    both("copy_pages", [m.P - 1, m.P - 2, -1, 2], [0, 1, 3, m.P])
    both("resize", [1, 8, 5, 4], [0, m.pt, 0, 0])
    both("compact")
    both("resize", [0, 1, 2, 3, 4, 5, 6, 7, 8], [0] * 9)
    # where a whole page ends at the fork, one append above meets a shared page (the model raises the same flag)
    assert c.flags() & ~TB_CACHE_SHARED == 0 and len(m.stack) == m.P


@pytest.mark.parametrize("seed", range(6))
def test_random_calls(seed):
    """Random lists with padding, numbers out of range, entries listed twice and more asked for than there is."""
    note(f"paged cache, random calls, seed {seed}")
    r = random.Random(seed)
    c, m = make(pages=r.choice([7, 40, 130]), pt=r.choice([1, 3, 8]), seqs=r.choice([3, 12, 33]), width=r.choice([1, 6, 17]),
                layout=r.choice(["token", "head"]))
    for step in range(40):
        n = r.randrange(0, m.S + 1)
        seqs = [r.randrange(-1, m.S + (r.random() < 0.1)) for _ in range(n)]
        if r.random() < 0.7:
            seqs = random.Random(step).sample(range(m.S), n)
        op = r.choice(["resize", "resize", "fork", "append", "compact", "copy_pages"])
        if op == "resize":
            lens = [r.choice([0, r.randrange(0, m.MP * m.pt + 1), m.lens[q] if 0 <= q < m.S else 0]) for q in seqs]
            if lens and r.random() < 0.1:
                lens[0] = r.choice([-1, m.MP * m.pt + 1])
            args = (seqs, lens)
        elif op == "fork":
            args = ([r.randrange(-1, m.S) for _ in seqs], seqs)
        elif op == "append":
            x = rows(c, 5, step)
            at = [(r.randrange(m.S), r.randrange(0, m.MP * m.pt)) for _ in range(20)]
            at = sorted(set(at))
            args = (x, [a for a, _ in at], [b for _, b in at], [r.randrange(5) for _ in at])
        elif op == "copy_pages":
            p = r.sample(range(m.P), 4)
            args = (p[:2], p[2:])
        else:
            args = ()
        getattr(c, op)(*[ints(a) if isinstance(a, list) else a.cuda() for a in args])
        getattr(m, op)(*args)
        m.check(c, f"step {step}: {op}")


@pytest.mark.parametrize("shape", [dict(pages=5000, pt=2, seqs=1500, width=9, heads=1, dim=4), dict(pages=70001, pt=1, seqs=40, width=6000, heads=1, dim=2)],
                         ids=str)
def test_many(shape):
    """Lists longer than a workgroup and scans over many chunks of pages."""
    note(f"paged cache, many entries, {shape}")
    c, m = make(**shape)
    r = random.Random(4)

    def both(name, *args):
        getattr(c, name)(*[ints(a) for a in args])
        getattr(m, name)(*args)
        m.check(c, name)

    half = list(range(0, m.S, 2))
    room = m.P // len(half) * m.pt
    lens = [min(r.randrange(1, m.MP * m.pt + 1), room) for _ in half]
    both("resize", half, lens)
    some = r.sample(half, len(half) // 3)
    both("fork", some + some[:5], list(range(1, m.S, 2))[:len(some)] + [m.S - 1 - 2 * k if m.S % 2 == 0 else m.S - 2 - 2 * k for k in range(5)])
    gone = r.sample(half, len(half) // 2)
    both("resize", gone, [r.choice([0, 1]) for _ in gone])
    both("compact")
    both("resize", list(range(m.S)), [0] * m.S)


def test_short_of_pages():
    note("paged cache, too few pages")
    from copy_reduce_amd import TB_CACHE_SHORT
    c, m = make(pages=6, pt=4)
    for name, args in (("resize", ([0, 1], [10, 9])), ("fork", ([0], [2])), ("resize", ([0, 1], [24, 1])), ("fork", ([0, 1], [3, 4])),
                       ("resize", ([1, 0], [28, 4])), ("fork", ([0], [5]))):
        getattr(c, name)(*[ints(a) for a in args])
        getattr(m, name)(*args)
        m.check(c, f"{name} {args}")
    assert c.flags(clear=True) & TB_CACHE_SHORT
    assert c.flags() == 0


def test_far_too_much_is_asked_for():
    """Sixteen rows of 2^28 pages: their sum is 0 in 32 bits."""
    note("paged cache, 2^32 pages asked for")
    require_gpu()
    from copy_reduce_amd.torch_api import PagedCache
    from copy_reduce_amd import _tb_cache as t
    rows, most = 16, 1 << 28
    c = PagedCache(torch.zeros(2, 5, 1, 1, 8, dtype=torch.bfloat16, device="cuda"), 1, rows, most)   # a table of 16 GiB
    c.resize(ints(list(range(rows))), ints([most] * rows))
    assert c.flags(clear=True) == t.TB_CACHE_SHORT
    assert not c.lens.any() and not c.refs.any() and int(c.counts[0]) == 5
    c.resize(ints([rows - 1]), ints([5]))
    assert c.flags() == 0 and c.table[rows - 1, :5].tolist() == [0, 1, 2, 3, 4] and int(c.counts[0]) == 0


@pytest.mark.parametrize("heads,dim,dtype,layout", [(3, 10, torch.bfloat16, "token"), (3, 10, torch.bfloat16, "head"), (2, 7, torch.uint8, "token"),
                                                    (3, 5, torch.float16, "head"), (4, 4, torch.uint8, "token"), (4, 4, torch.uint8, "head")])
@pytest.mark.parametrize("pools", [1, 4, 7])
def test_append_by_every_width(heads, dim, dtype, layout, pools):
    """Tokens and heads of 16, 4 and fewer bytes, and rows that begin at odd places."""
    note(f"paged cache, append {heads} x {dim} {dtype} {layout} {pools} pools")
    require_gpu()
    from copy_reduce_amd.torch_api import PagedCache
    pt, n = 3, 8
    page = (pt, heads, dim) if layout == "token" else (heads, pt, dim)
    kv = torch.zeros((pools, 6) + page, dtype=dtype, device="cuda")
    c = PagedCache(kv, pt, 2, 4, layout=layout)
    c.resize(ints([1]), ints([n]))
    for shift in (0, 1, 2, 8):
        flat = torch.randint(1, 100, (shift + pools * (n + 1) * heads * dim,), device="cuda").to(dtype)
        x = flat[shift:].view(pools, n + 1, heads, dim)
        kv.zero_()
        c.append(x, ints([1] * n), ints(list(range(n))), ints([n - i for i in range(n)]))
        by_token = kv if layout == "token" else kv.transpose(2, 3)
        for i in range(n):
            assert torch.equal(by_token[:, int(c.table[1, i // pt]), i % pt], x[:, n - i]), (shift, i)
        assert int((kv != 0).sum()) == pools * n * heads * dim
    assert c.flags() == 0


def test_append_of_more_pieces_than_a_grid_has_threads():
    """2^32 and more pieces of 16 bytes: a million tokens of 64 KiB, of few rows, to few positions."""
    note("paged cache, append of 64 GiB")
    require_gpu()
    from copy_reduce_amd.torch_api import PagedCache
    n, pt = (1 << 20) + 5, 4
    kv = torch.zeros(1, 3, pt, 256, 128, dtype=torch.bfloat16, device="cuda")
    c = PagedCache(kv, pt, 1, 3)
    c.resize(ints([0]), ints([9]))
    x = torch.randn(1, 9, 256, 128, device="cuda").to(torch.bfloat16)
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    pos[-9:] = torch.arange(9, dtype=torch.int32, device="cuda")
    c.append(x, torch.zeros_like(pos), pos, pos)
    table = c.table[0].tolist()
    for i in range(9):
        assert torch.equal(kv[0, table[i // pt], i % pt], x[0, i]), i
    assert c.flags() == 0


def test_shared_pages_are_not_written():
    note("paged cache, append to a shared page")
    from copy_reduce_amd import TB_CACHE_SHARED
    c, m = make(pt=4)
    c.resize(ints([0]), ints([8])), m.resize([0], [8])
    c.fork(ints([0]), ints([1])), m.fork([0], [1])
    x = rows(c, 2)
    c.append(x.cuda(), ints([1, 0]), ints([3, 7])), m.append(x, [1, 0], [3, 7])
    m.check(c, "append")
    assert c.flags() == TB_CACHE_SHARED


def test_copy_between_caches():
    note("paged cache, pages from another cache")
    c, m = make(pages=9, pad=8)
    d, n = make(pages=31)
    c.copy_pages(ints([8, 0, 3]), ints([30, 2, 2]), src=d)
    m.copy_pages([8, 0, 3], [30, 2, 2], other=n)
    m.check(c, "destination")
    n.check(d, "source")


def test_more_pools_than_one_launch_takes():
    note("paged cache, 130 pools")
    c, m = make(pages=8, pt=2, heads=1, layers=65)
    for name, args in (("resize", ([0], [3])), ("fork", ([0], [1])), ("copy_pages", ([5], [0])), ("resize", ([0], [0])), ("compact", ())):
        getattr(c, name)(*[ints(a) for a in args])
        getattr(m, name)(*args)
    x = rows(c, 1)
    c.append(x.cuda(), ints([1]), ints([2])), m.append(x, [1], [2])
    m.check(c, "130 pools")


def test_no_pools_and_two_pages():
    """The bookkeeping alone, through the C call; the smallest caches."""
    note("paged cache, no pools")
    import copy_reduce_amd as tb
    c, m = make(pages=2, pt=2, seqs=3, width=2)
    c._c.npools = 0
    a, b = ints([0]), ints([3])
    s = torch.cuda.current_stream().cuda_stream
    for name, args in (("resize", ([0], [2])), ("fork", ([0], [2])), ("resize", ([0], [0])), ("compact", ()), ("resize", ([2], [0]))):
        getattr(c, name)(*[ints(x) for x in args])
        getattr(m, name)(*args)
        m.check(c, name)
    assert tb.lib.tb_page_append(c._c, a.data_ptr(), 1, 32, 32, a.data_ptr(), b.data_ptr(), None, 1, s) == tb.TB_OK
    c, m = make(pages=1, pt=2, seqs=1, width=1)
    for name, args in (("resize", ([0], [2])), ("compact", ()), ("resize", ([0], [1])), ("resize", ([0], [0])), ("compact", ())):
        getattr(c, name)(*[ints(x) for x in args])
        getattr(m, name)(*args)
        m.check(c, name)


def test_far_pages():
    """Byte offsets past 2^32 within one pool."""
    note("paged cache, a pool of 5.9 GiB")
    require_gpu()
    from copy_reduce_amd.torch_api import PagedCache
    pages, pt = 3000, 16
    kv = torch.zeros(2, pages, pt, 8, 8192, dtype=torch.bfloat16, device="cuda")
    c = PagedCache(kv, pt, 2, 4)
    c.free_list[:pages] = torch.arange(pages, dtype=torch.int32, device="cuda")   # highest page on top
    c.resize(ints([0]), ints([20]))
    x = torch.randn(2, 20, 8, 8192, device="cuda").to(torch.bfloat16)
    c.append(x, ints([0] * 20), ints(list(range(20))))
    assert torch.equal(kv[:, pages - 1], x[:, :16]) and torch.equal(kv[:, pages - 2, :4], x[:, 16:])
    c.fork(ints([0]), ints([1]))
    assert torch.equal(kv[:, pages - 3, :4], x[:, 16:]) and not kv[:, pages - 3, 4:].any()
    c.copy_pages(ints([pages - 4, 0]), ints([pages - 1, pages - 1]))
    assert torch.equal(kv[:, pages - 4], x[:, :16])
    c.compact()
    assert torch.equal(kv[:, 2], x[:, :16]) and c.table[0, :2].tolist() == [2, 1] and c.table[1, :2].tolist() == [2, 0]


def test_captured_step_replays():
    """A step of every call in one graph, replayed with eager work in between."""
    note("paged cache, captured step")
    c, m = make(pages=64, pt=4, seqs=8, width=8)
    x = rows(c, 6, 3)
    xs, seqs, lens, at = x.cuda(), ints([0, 1]), ints([5, 6]), ints([3, 4, 5, 0, 1, 2])
    grow, kids, owner = ints([6, 9]), ints([2, 3]), ints([0, 0, 0, 1, 1, 1])

    zero = ints([0, 0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            c.resize(seqs, lens), c.append(xs, owner, at), c.fork(seqs, kids), c.resize(seqs, grow), c.compact(), c.resize(kids, zero)
    torch.cuda.current_stream().wait_stream(s)
    m.check(c, "captured, not run")
    for k in range(4):
        graph.replay()
        m.resize([0, 1], [5, 6]), m.append(x, [0, 0, 0, 1, 1, 1], [3, 4, 5, 0, 1, 2]), m.fork([0, 1], [2, 3])
        m.resize([0, 1], [6, 9]), m.compact(), m.resize([2, 3], [0, 0])
        m.check(c, f"replay {k}")
        c.resize(ints([5, 0]), ints([k + 1, 2])), m.resize([5, 0], [k + 1, 2])
        torch.cuda.synchronize()
        m.check(c, f"eager after replay {k}")


def test_on_a_given_stream():
    note("paged cache, another stream")
    c, m = make()
    s = torch.cuda.Stream()
    a, b = ints([0, 1]), ints([7, 9])
    torch.cuda.synchronize()
    c.resize(a, b, stream=s), m.resize([0, 1], [7, 9])
    c.free(a[:1], stream=s), m.resize([0], [0])
    s.synchronize()
    m.check(c, "resize on a stream")


def test_timing_hook_spans_a_call():
    """The launch-carried events of a call of several kernels: start before the first, stop after the last."""
    note("paged cache, launch events")
    torch_ = require_gpu()
    import copy_reduce_amd as tb
    c, m = make()
    e0, e1 = torch_.cuda.Event(enable_timing=True), torch_.cuda.Event(enable_timing=True)
    e0.record(), e1.record()
    torch_.cuda.synchronize()
    for name, args in (("resize", ([0], [9])), ("fork", ([0], [1])), ("compact", ())):
        listed = [ints(a) for a in args]
        tb.tb_time_next_launch(e0.cuda_event, e1.cuda_event)
        getattr(c, name)(*listed)
        getattr(m, name)(*args)
        torch_.cuda.synchronize()
        assert e0.elapsed_time(e1) > 0
        m.check(c, name)


def test_refusals():
    note("paged cache, refusals")
    c, _ = make()
    from copy_reduce_amd import TBError
    from copy_reduce_amd.torch_api import PagedCache
    with pytest.raises(ValueError):
        c.resize(torch.zeros(1, dtype=torch.int64, device="cuda"), ints([0]))
    with pytest.raises(ValueError):
        c.resize(ints([0]), ints([0, 1]))
    with pytest.raises(ValueError):
        c.fork(ints([0, 1, 2, 3])[::2], ints([4, 5]))
    with pytest.raises(ValueError):
        c.fork(torch.zeros(1, dtype=torch.int32), ints([0]))
    with pytest.raises(TBError):
        c.resize(ints([0] * 10), ints([0] * 10))           # more entries than rows
    with pytest.raises(ValueError):
        c.append(rows(c, 1).cuda().float(), ints([0]), ints([0]))
    with pytest.raises(ValueError):
        c.append(rows(c, 1).cuda(), ints([0, 1]), ints([0, 0]))
    with pytest.raises(ValueError):
        c.append(rows(c, 1)[:1].cuda(), ints([0]), ints([0]))
    with pytest.raises(ValueError):
        PagedCache(torch.zeros(2, 8, 4, 2, 8, device="cuda"), 8, 2, 2)
    with pytest.raises(ValueError):
        PagedCache(torch.zeros(2, 8, 4, 2, 8, device="cuda").transpose(3, 4), 4, 2, 2)
    with pytest.raises(ValueError):
        PagedCache(torch.zeros(2, 8, 4, 2, 8, device="cuda"), 4, 2, 2, state=torch.zeros(3, dtype=torch.int32, device="cuda"))
