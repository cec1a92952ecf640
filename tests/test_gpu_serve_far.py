"""GPU tests of the serving step's calls at the ends of their ranges: positions near 2^31, pools of 16 GiB, rows at odd places.
The bounds of the attention are those of test_gpu_tree_attention.py."""
import math

import pytest
import torch

from gpu_util import note, require_gpu
from serve_model import decode, encode, head_bytes
from test_gpu_tree_attention import compare, inputs, ints

pytestmark = pytest.mark.gpu


def far_cache(pt, width, heads, dim, dtype, layout, fp4, seqs=2, pages=3, seed=0):
    """A cache whose rows refer to the same few pages again and again, so that sequences of 2^31 tokens take no memory; what
    the pages hold as numbers [2, pages, pt, heads, dim], and the pages of a row."""
    require_gpu()
    from copy_reduce_amd.torch_api import PagedCache
    g = torch.Generator().manual_seed(seed)
    held = torch.randn(2, pages, pt, heads, dim, generator=g).to(dtype)
    raw = held
    if fp4:
        raw = encode(held)
        held = decode(raw, dim).to(dtype)
    pools = raw if layout == "token" else raw.transpose(2, 3).contiguous()
    c = PagedCache(pools.cuda(), pt, seqs, width, layout=layout, fp4=dtype if fp4 else None)
    row = torch.randint(0, pages, (width,), generator=g, dtype=torch.int32)
    c.table.copy_(row.cuda().expand(seqs, width))
    c.refs.fill_(1)
    return c, held, row, g


def context(held, row, pool, tokens):
    """[tokens, heads, dim] in 64 bits."""
    pt = held.shape[2]
    tokens = torch.as_tensor(tokens, dtype=torch.int64)
    return held[pool, row[tokens // pt].long(), tokens % pt].double()


def definition(held, row, q, k, v, lens, window, sinks):
    """Chains over the last tokens and the sinks: (out, lse, A, S, V) as the models give them."""
    b, t, hq, d = q.shape
    group = hq // k.shape[2]
    out, lse = torch.zeros(b, t, hq, d, dtype=torch.float64), torch.zeros(b, t, hq, dtype=torch.float64)
    a, s, big = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(lse)
    for i, n in enumerate(lens):
        for x in range(t):
            at = sorted(set(range(min(sinks, n))) | set(range(max(0, n + x + 1 - window), n)))
            sees = [u for u in range(x + 1) if x - u < window or n + u < sinks]
            key = torch.cat([context(held, row, 0, at), k[i, sees].double()])
            val = torch.cat([context(held, row, 1, at), v[i, sees].double()])
            for h in range(hq):
                qq, kk, vv = q[i, x, h].double(), key[:, h // group], val[:, h // group]
                y = kk @ qq / math.sqrt(d)
                z = torch.logsumexp(y, 0)
                w = torch.exp(y - z)
                out[i, x, h], lse[i, x, h], a[i, x, h] = w @ vv, z, w @ vv.abs()
                s[i, x, h], big[i, x, h] = (kk.abs() @ qq.abs()).max() / math.sqrt(d), vv.abs().max()
    return out, lse, a, s, big


@pytest.mark.parametrize("fp4", [False, True], ids=["16 bits", "4 bits"])
@pytest.mark.parametrize("layout,pt,width", [("token", 65536, 32767), ("head", 65521, 32775), ("token", 1021, 2103313)])
def test_windows_near_2_31(layout, pt, width, fp4):
    """Few rows and many, by whole sequences (a window of 40) and by shares (of 2,500)."""
    note(f"windows at positions near 2^31, pages of {pt}, {layout}, 4 bits {fp4}")
    from copy_reduce_amd.torch_api import tree_attention
    assert 2 ** 31 - 2 ** 17 < pt * width < 2 ** 31
    c, held, row, g = far_cache(pt, width, 2, 64, torch.bfloat16, layout, fp4)
    lens = [pt * width, pt * width - pt // 2]
    c.lens.copy_(ints(lens))
    for t, window, sinks in ((1, 40, 3), (5, 40, 0), (40, 30, 5), (1, 2500, 2), (40, 2500, 2)):
        q, k, v = inputs(g, 2, t, 4, 2, 64, torch.bfloat16)
        got = tree_attention(q.cuda(), k.cuda(), v.cuda(), c, 0, ints([0, 1]), window=window, sinks=sinks)
        compare(got, definition(held, row, q, k, v, lens, window, sinks), window + sinks + t, 64, q.dtype, f"{t} nodes, window {window}")


def test_sinks_near_2_31_and_windows_of_2_32():
    """Sinks past the context, and a window as wide as can be said, over a short sequence of a long row."""
    note("sinks of 2^32 - 1")
    from copy_reduce_amd.torch_api import tree_attention
    c, held, row, g = far_cache(1024, 2097151, 1, 64, torch.bfloat16, "token", False)
    c.lens.copy_(ints([300, 7]))
    q, k, v = inputs(g, 2, 20, 2, 1, 64, torch.bfloat16)
    for window, sinks in ((3, 2 ** 32 - 1), (2 ** 32 - 1, 2 ** 32 - 1), (2 ** 32 - 1, 0), (3, 310)):
        got = tree_attention(q.cuda(), k.cuda(), v.cuda(), c, 0, ints([0, 1]), window=window, sinks=sinks)
        compare(got, definition(held, row, q, k, v, [300, 7], window, sinks), 320, 64, q.dtype, f"window {window}, sinks {sinks}")


@pytest.mark.parametrize("fp4", [False, True], ids=["16 bits", "4 bits"])
@pytest.mark.parametrize("layout,pt,width", [("token", 65536, 32767), ("head", 65521, 32775)])
def test_append_and_read_near_2_31(layout, pt, width, fp4):
    note(f"append and read near 2^31, pages of {pt}, {layout}, 4 bits {fp4}")
    c, held, row, g = far_cache(pt, width, 2, 64, torch.float16, layout, fp4)
    n = pt * width
    c.lens.copy_(ints([n, 0]))
    at = [n - 1, n - pt, n - pt - 1, 0, 2 ** 30, 2 ** 30 + 1]
    places = {(int(row[p // pt]), p % pt) for p in at}
    at = at if len(places) == len(at) else at[:2]
    new = torch.randn(2, len(at), 2, 64, generator=g).to(torch.float16)
    c.append(new.cuda(), ints([0] * len(at)), ints(at))
    got = c.read(ints([0] * len(at)), ints(at)).cpu()
    assert torch.equal(got, decode(encode(new), 64).to(torch.float16) if fp4 else new)
    others = [p for p in (5, n - 100, 2 ** 30 + 7, 2 ** 31 - 2 ** 18) if (int(row[p // pt]), p % pt) not in places]
    got = c.read(ints([0] * len(others)), ints(others)).cpu()
    for pool in range(2):
        assert torch.equal(got[pool].double(), context(held, row, pool, others))
    assert c.flags() == 0
    c.read(ints([0, 0]), ints([n, 2 ** 31 - 1]))
    assert c.flags() == 2


@pytest.mark.parametrize("fp4", [False, True], ids=["16 bits", "4 bits"])
def test_pages_4_gib_apart(fp4):
    """In 4 bits the largest pool that the attention reads, 16 GiB: the places of its last page's tokens are near 2^32 words."""
    note(f"pools of 16 GiB, 4 bits {fp4}")
    require_gpu()
    from copy_reduce_amd.torch_api import PagedCache, tree_attention
    g = torch.Generator().manual_seed(1)
    pages, pt, heads, dim = 4, 32, 2, 128
    each = head_bytes(dim) if fp4 else dim
    apart = (1 << 32) // (1 if fp4 else 2)
    dtype = torch.uint8 if fp4 else torch.bfloat16
    room = [torch.empty(pages * apart, dtype=dtype, device="cuda") for _ in range(2)]
    pools = [r.as_strided((pages, pt, heads, each), (apart, heads * each, each, 1)) for r in room]
    c = PagedCache(pools, pt, 2, pages, fp4=torch.bfloat16 if fp4 else None)
    c.resize(ints([1]), ints([pages * pt]))
    n = pages * pt
    new = torch.randn(2, n, heads, dim, generator=g).to(torch.bfloat16)
    where = torch.randperm(n, generator=g).tolist()
    c.append(new.cuda(), ints([1] * n), ints(where))
    held = decode(encode(new), dim).to(torch.bfloat16) if fp4 else new
    assert torch.equal(c.read(ints([1] * n), ints(where)).cpu(), held)
    by_position = torch.empty_like(held)
    by_position[:, where] = held
    row = torch.arange(pages, dtype=torch.int32)
    by_page = by_position.view(2, pages, pt, heads, dim)
    for t in (1, 20):
        q, k, v = inputs(g, 1, t, 4, heads, dim, torch.bfloat16)
        for window, sinks in ((None, 0), (50, 3)):
            got = tree_attention(q.cuda(), k.cuda(), v.cuda(), c, 0, ints([1]), window=window, sinks=sinks)
            compare(got, definition(by_page, row, q, k, v, [n], window or 10 ** 6, sinks), n + t, dim, q.dtype, f"{t} nodes, window {window}")
    assert c.flags() == 0


@pytest.mark.parametrize("fp4", [False, True], ids=["16 bits", "4 bits"])
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("dim,heads", [(64, 1), (96, 3), (128, 2)])
@pytest.mark.parametrize("off,gap", [(1, 0), (3, 1), (0, 5), (2, 2)])
def test_rows_at_odd_places(dim, heads, layout, off, gap, fp4):
    """Rows that begin at any element, with any number of elements between them: what lies between stays as it was."""
    note(f"rows {off} elements on, {gap} apart, dim {dim}, {heads} heads, {layout}, 4 bits {fp4}")
    require_gpu()
    from copy_reduce_amd.torch_api import PagedCache
    g = torch.Generator().manual_seed(dim + off)
    pt, n, size = 8, 21, heads * dim
    page = (pt, heads) if layout == "token" else (heads, pt)
    pools = torch.zeros((2, 6) + page + (head_bytes(dim) if fp4 else dim,), dtype=torch.uint8 if fp4 else torch.bfloat16, device="cuda")
    c = PagedCache(pools, pt, 1, 6, layout=layout, fp4=torch.bfloat16 if fp4 else None)
    c.resize(ints([0]), ints([n]))
    new = torch.randn(2, n, heads, dim, generator=g).to(torch.bfloat16)

    def room():
        whole = torch.full((off + 2 * n * (size + gap) + 7,), 77.0, dtype=torch.bfloat16, device="cuda")
        return whole, whole.as_strided((2, n, heads, dim), (n * (size + gap), size + gap, dim, 1), off)

    _, rows = room()
    rows.copy_(new)
    order = torch.randperm(n, generator=g).tolist()
    c.append(rows, ints([0] * n), ints(order))
    whole, out = room()
    c.read(ints([0] * n), ints(order), out=out)
    assert torch.equal(out.cpu(), decode(encode(new), dim).to(torch.bfloat16) if fp4 else new)
    out.fill_(77.0)
    assert bool((whole == 77).all()) and c.flags() == 0
