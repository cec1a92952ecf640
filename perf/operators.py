"""Cases of the paged key/value cache and of the attention of drafted tokens over it.

A cache is a tensor of pools, keys and values of each layer in turn, every pool a run of pages of a few tokens. Its bookkeeping is one int32
tensor: table (sequence, position -> page), lens (tokens of a sequence), refs (references to a page), free (a stack of free pages), counts (their
number, flags). The operators that change the bookkeeping start each pass from the copy that the scheduler holds.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}

# Pools of 16 KiB pages (8 tokens of 8 heads of 128 in 16 bits) in a 4 GiB cache are what the transfer workloads write into.
LISTED = [
    # accepted tokens of a few short sequences into a two-layer cache laid out by head: a call whose cost is its launch
    {"name": "append_small", "op": "append", "n": 13, "seqs": 5, "ctx": 90, "pools": 4, "pt": 16, "heads": 3, "dim": 64, "layout": "head", "dtype": "fp16"},
    # pages moved in a 4 GiB cache of 32 layers, as for prefixes that are kept elsewhere
    {"name": "copy_pages_16k", "op": "copy", "n": 400, "pages": 4096, "pools": 64, "pt": 8, "heads": 8, "dim": 128, "layout": "token", "dtype": "bf16"},
    # one prompt sampled three ways
    {"name": "fork_one_prompt", "op": "fork", "parents": 1, "ways": 3, "ctx": 701, "pools": 8, "pt": 16, "heads": 2, "dim": 64, "layout": "token", "dtype": "bf16"},
    # candidates of a whole batch, laid out by head
    {"name": "fork_batch", "op": "fork", "parents": 48, "ways": 4, "ctx": 2001, "pools": 32, "pt": 16, "heads": 8, "dim": 128, "layout": "head", "dtype": "bf16"},
    # a small cache tidied between requests, odd page size
    {"name": "compact_small", "op": "compact", "seqs": 9, "ctx": 333, "free": 0.5, "move": 0.2, "pools": 4, "pt": 5, "heads": 3, "dim": 32, "layout": "token", "dtype": "fp16"},
    # a 4 GiB cache before a transfer of large blocks
    {"name": "compact_4gib", "op": "compact", "seqs": 64, "ctx": 900, "free": 0.1, "move": 0.15, "pools": 64, "pt": 8, "heads": 8, "dim": 128, "layout": "token", "dtype": "bf16"},
    # a few requests end, a few begin
    {"name": "free_few", "op": "resize", "seqs": 16, "listed": 6, "ctx": 500, "spare": 1.0, "pools": 2, "pt": 16, "heads": 1, "dim": 8, "layout": "token", "dtype": "bf16"},
    # a large batch turns over: long sequences freed and admitted at once
    {"name": "free_batch", "op": "resize", "seqs": 512, "listed": 511, "ctx": 16000, "spare": 1.0, "pools": 2, "pt": 16, "heads": 1, "dim": 8, "layout": "token", "dtype": "bf16"},
    # single tokens of a few short sequences
    {"name": "decode_short", "op": "attention", "batch": 4, "nodes": 1, "tree": False, "ctx": 333, "groups": 4, "pt": 16, "heads": 2, "dim": 64, "layout": "head", "dtype": "fp16"},
    # single tokens of a large ragged batch: the cache's bytes decide
    {"name": "decode_64", "op": "attention", "batch": 64, "nodes": 1, "tree": False, "ctx": 8191, "groups": 4, "pt": 16, "heads": 8, "dim": 128, "layout": "token", "dtype": "bf16"},
    # small trees with odd heads, head size and pages
    {"name": "tree_13", "op": "attention", "batch": 7, "nodes": 13, "tree": True, "ctx": 2047, "groups": 7, "pt": 20, "heads": 4, "dim": 96, "layout": "token", "dtype": "fp16"},
    # wide trees over long contexts: products count as much as bytes
    {"name": "tree_64", "op": "attention", "batch": 16, "nodes": 64, "tree": True, "ctx": 16383, "groups": 4, "pt": 32, "heads": 8, "dim": 128, "layout": "token", "dtype": "bf16"},
]


def listed():
    return [dict(c) for c in LISTED]


def _log(rng, a, b):
    return min(b, max(a, int(round(math.exp(rng.uniform(math.log(a), math.log(b + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "copy", "fork", "compact", "resize", "attention", "attention", "attention"])
    c = {"op": op, "layout": rng.choice(["token", "head"]), "dtype": rng.choice(["bf16", "fp16"]), "pt": rng.choice([1, 5, 8, 16, 16, 20, 32, 64])}
    if op == "attention":
        while True:
            c.update(batch=_log(rng, 1, 64), nodes=rng.choice([1, 1, _log(rng, 2, 100), _log(rng, 2, 100)]), ctx=_log(rng, 1, 20000), groups=rng.choice([1, 2, 4, 5, 7, 8, 16]),
                     heads=rng.choice([1, 2, 3, 4, 8]), dim=rng.choice([64, 96, 128, 128, 256]), tree=rng.random() < 0.7)
            keys = c["batch"] * c["heads"] * c["dim"] * (c["ctx"] + c["nodes"])
            if keys <= 16 * 8 * 128 * 16384 and keys * c["nodes"] * c["groups"] <= 16 * 8 * 128 * 16384 * 256:
                c["tree"] = c["tree"] and c["nodes"] > 1
                return c
    while True:
        c.update(pools=2 * _log(rng, 1, 32), heads=rng.choice([1, 2, 3, 4, 8]), dim=rng.choice([32, 64, 96, 128, 256]))
        if op == "copy":
            c.update(n=_log(rng, 1, 2000), pages=0)
            c["pages"] = 2 * c["n"] + rng.randrange(1, 100)
        elif op == "append":
            c.update(n=_log(rng, 1, 4000), seqs=_log(rng, 1, 100), ctx=_log(rng, 1, 2000))
        elif op == "fork":
            c.update(parents=_log(rng, 1, 100), ways=rng.choice([1, 2, 3, 4]), ctx=_log(rng, 1, 4000))
        elif op == "compact":
            c.update(seqs=_log(rng, 1, 100), ctx=_log(rng, 1, 4000), free=rng.uniform(0.1, 0.9), move=rng.uniform(0.0, 0.4))
        else:
            c.update(seqs=_log(rng, 2, 512), ctx=_log(rng, 2, 16000), spare=rng.uniform(0.5, 1.5), pools=2, heads=1, dim=8)
            c["listed"] = rng.randrange(1, c["seqs"] + 1)
            return c
        if c["pools"] * _pages(c) * _page(c) <= 1 << 32:
            return c


def _lens(n, ctx):
    return [max(1, (i + 1) * ctx // n) for i in range(n)]


def _npg(length, pt):
    return -(-length // pt)


def _token(c):
    return 2 * c["heads"] * c["dim"]


def _page(c):
    return _token(c) * c["pt"]


def _rows(c):
    """Sequences that the table has room for."""
    return {"copy": 1, "append": c.get("seqs"), "compact": c.get("seqs"), "resize": c.get("seqs"), "fork": c.get("parents", 0) * (1 + c.get("ways", 0)),
            "attention": c.get("batch")}[c["op"]]


def _used(c):
    """The lengths that the sequences have before the call."""
    if c["op"] == "copy":
        return []
    if c["op"] == "resize":  # every third one is yet to begin
        return [0 if i % 3 == 2 else v for i, v in enumerate(_lens(c["seqs"], c["ctx"]))]
    return _lens({"fork": c.get("parents"), "attention": c.get("batch")}.get(c["op"], c.get("seqs")), c["ctx"])


def _live(c):
    return sum(_npg(v, c["pt"]) for v in _used(c))


def _pages(c):
    """Pages of the cache."""
    if c["op"] == "copy":
        return c["pages"]
    if c["op"] == "fork":
        return _live(c) + c["parents"] * c["ways"] + 7
    if c["op"] == "compact":
        return int(_live(c) * (1 + c["free"])) + 2
    if c["op"] == "resize":  # room for whatever the listed ones grow to
        return _live(c) + int(c["seqs"] * _npg(c["ctx"], c["pt"]) * c["spare"]) + c["seqs"] * _npg(c["ctx"], c["pt"])
    return _live(c) + 3


def _moved(c):
    live, pages = _live(c), _pages(c)
    return min(int(live * c["move"]), pages - live)


def _views(book, rows, width, pages):
    a = rows * width
    return {"table": book[:a].view(rows, width), "lens": book[a:a + rows], "refs": book[a + rows:a + rows + pages],
            "free": book[a + rows + pages:a + rows + 2 * pages], "counts": book[a + rows + 2 * pages:a + rows + 2 * pages + 4]}


def _filled(shape, dtype, g, dev):
    t = torch.empty(shape, dtype=dtype, device=dev)
    return t.normal_(generator=g)


def prepare(case, seed):
    c, dev = case, torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    pt, rows, pages, dtype = c["pt"], _rows(c), _pages(c), DTYPES[c["dtype"]]
    used = _used(c)
    order = torch.randperm(len(used), generator=h).tolist() if c["op"] != "resize" else list(range(len(used)))
    lens = [0] * rows
    for i, j in enumerate(order):
        lens[i] = used[j]
    width = max(1, _npg(c.get("ctx", 1), pt) + 1)
    pools = c.get("pools", 2)
    page = (pt, c["heads"], c["dim"]) if c["layout"] == "token" else (c["heads"], pt, c["dim"])
    kv = _filled((pools, pages) + page, dtype, g, dev)

    # pages: at random places of the cache, or (to be compacted) a given number of them above the live ones' count
    live = _live(c)
    if c["op"] == "compact":
        m = _moved(c)
        low = torch.randperm(live, generator=h)[:live - m]
        high = live + torch.randperm(pages - live, generator=h)[:m]
        at = torch.cat([low, high])[torch.randperm(live, generator=h)]
    else:
        at = torch.randperm(pages, generator=h)[:live]
    n = torch.tensor([_npg(v, pt) for v in lens], dtype=torch.int64).reshape(-1)
    j = torch.arange(width)
    table = torch.zeros(rows, width, dtype=torch.int64)
    table[j < n[:, None]] = at
    refs = torch.zeros(pages, dtype=torch.int64)
    refs[at] = 1
    if c["op"] == "resize" and rows > 4:  # the second sequence's copy is the fourth's beginning: pages with two references
        k = int(min(n[1], n[3], 3))
        refs[table[3, :k]] = 0
        table[3, :k] = table[1, :k]
        refs[table[3, :k]] = 2
    empty = torch.nonzero(refs == 0).flatten()
    empty = empty[torch.randperm(len(empty), generator=h)]
    free = torch.zeros(pages, dtype=torch.int64)
    free[:len(empty)] = empty
    book = torch.cat([table.flatten(), torch.tensor(lens, dtype=torch.int64), refs, free, torch.tensor([len(empty), 0, 0, 0])]).to(torch.int32).to(dev)
    s = {"case": c, "kv": kv, "held": book, "book": book.clone(), "shape": (rows, width, pages)}

    def ints(v):
        return torch.as_tensor(v, dtype=torch.int32).to(dev)

    if c["op"] == "copy":
        p = torch.randperm(pages, generator=h)
        src, dst = p[:c["n"]].clone(), p[c["n"]:2 * c["n"]].clone()
        src[-1] = src[0]  # one page to two places
        s.update(src=ints(src), dst=ints(dst))
    elif c["op"] == "append":
        # the last tokens of the sequences, a few of those that were drafted; one in eight is padding
        tok = torch.cat([torch.stack([torch.full((v,), i), torch.arange(v)], 1) for i, v in enumerate(lens)])
        tok = tok[torch.randperm(len(tok), generator=h)[:c["n"]]]
        seqs = tok[:, 0].clone()
        seqs[7::8] = -1
        drafted = 2 * len(tok) + 1
        s.update(seqs=ints(seqs), at=ints(tok[:, 1]), index=ints(torch.randperm(drafted, generator=h)[:len(tok)]),
                 new=_filled((pools, drafted, c["heads"], c["dim"]), dtype, g, dev))
    elif c["op"] == "fork":
        kids = torch.randperm(c["parents"] * c["ways"], generator=h) + c["parents"]
        s.update(parents=ints(torch.arange(c["parents"]).repeat(c["ways"])), children=ints(kids))
    elif c["op"] == "resize":
        pick = torch.arange(c["listed"])[torch.randperm(c["listed"], generator=h)]
        now = torch.tensor(lens)[pick]
        step = torch.randint(1, max(2, c["ctx"]), (c["listed"],), generator=h)
        end = torch.where(pick % 3 == 0, torch.zeros_like(now), torch.where(pick % 3 == 1, torch.clamp(now + 1 + step % 9, max=c["ctx"]), torch.clamp(step, max=c["ctx"])))
        s.update(seqs=ints(pick), to=ints(end))
    elif c["op"] == "attention":
        b, t, hk, hq, d = c["batch"], c["nodes"], c["heads"], c["heads"] * c["groups"], c["dim"]
        s.update(q=_filled((b, t, hq, d), dtype, g, dev), k=_filled((b, t, hk, d), dtype, g, dev), v=_filled((b, t, hk, d), dtype, g, dev),
                 seqs=ints(torch.randperm(rows, generator=h)), mask=None, nodes=None)
        if c["tree"]:
            # a node's parent is any earlier node; in every third tree the last nodes are padding
            parent = (torch.rand(b, t, generator=h) * torch.arange(t)).long()
            sees = torch.zeros(b, t, t, dtype=torch.bool)
            sees[:, 0, 0] = True
            for i in range(1, t):
                sees[:, i] = sees[torch.arange(b), parent[:, i]]
                sees[:, i, i] = True
            words = -(-t // 64)
            bits = torch.zeros(b, t, words * 64, dtype=torch.int64)
            bits[..., :t] = sees
            one = torch.ones((), dtype=torch.int64) << torch.arange(64)
            s["mask"] = (bits.view(b, t, words, 64) * one).sum(-1).to(dev)
            s["nodes"] = ints([t - t // 3 if i % 3 == 2 else t for i in range(b)])
    if own:
        from copy_reduce_amd.torch_api import PagedCache, tree_attention, tree_attention_workspace
        s["cache"] = PagedCache(kv, page_tokens=pt, max_seqs=rows, max_pages=width, layout=c["layout"], state=s["book"])
        if c["op"] == "attention":
            s.update(attend=tree_attention, workspace=tree_attention_workspace(s["q"], s["cache"]))
    return s


def run(state):
    op = state["case"]["op"]
    if op in ("fork", "compact", "resize"):
        state["book"].copy_(state["held"])  # the scheduler's tables
    if own:
        cache = state["cache"]
        if op == "copy":
            cache.copy_pages(state["dst"], state["src"])
        elif op == "append":
            cache.append(state["new"], state["seqs"], state["at"], index=state["index"])
        elif op == "fork":
            cache.fork(state["parents"], state["children"])
        elif op == "compact":
            cache.compact()
        elif op == "resize":
            cache.resize(state["seqs"], state["to"])
        else:
            out, lse = state["attend"](state["q"], state["k"], state["v"], cache, 0, state["seqs"], mask=state["mask"], nodes=state["nodes"], workspace=state["workspace"])
            return {"out": out, "lse": lse}
    elif op == "attention":
        return _attention(state)
    else:
        {"copy": _copy, "append": _append, "fork": _fork, "compact": _compact, "resize": _resize}[op](state)
    return {"book": state["book"]} if op == "resize" else {"kv": state["kv"]} if op in ("copy", "append") else {"kv": state["kv"], "book": state["book"]}


def _copy(s):
    s["kv"][:, s["dst"].long()] = s["kv"][:, s["src"].long()]


def _append(s):
    b = _views(s["book"], *s["shape"])
    pt = s["case"]["pt"]
    there = s["seqs"] >= 0
    q, at, x = s["seqs"][there].long(), s["at"][there].long(), s["index"][there].long()
    page = b["table"][q, at // pt].long()
    by_token = s["kv"] if s["case"]["layout"] == "token" else s["kv"].transpose(2, 3)
    by_token[:, page, at % pt] = s["new"][:, x]


def _fork(s):
    b, pt, kv = _views(s["book"], *s["shape"]), s["case"]["pt"], s["kv"]
    par, kid = s["parents"].long(), s["children"].long()
    length = b["lens"][par]
    full, rest = length // pt, length % pt
    need = (rest > 0).to(torch.int32)
    rank = torch.cumsum(need, 0) - need
    page = b["free"][(b["counts"][0] - 1 - rank).clamp(min=0)]
    j = torch.arange(s["shape"][1], device=kv.device)
    theirs, shared = b["table"][par], j < full[:, None]
    tail = (j == full[:, None]) & (need[:, None] > 0)
    b["table"][kid] = torch.where(shared, theirs, torch.where(tail, page[:, None], b["table"][kid]))
    b["refs"].index_add_(0, theirs.flatten(), shared.flatten().to(torch.int32))
    b["refs"].index_add_(0, page, need)
    b["lens"][kid] = length
    b["counts"][0] -= need.sum().to(torch.int32)
    with_tail = torch.nonzero(need).flatten()
    src = theirs[with_tail, full[with_tail].long()].long()
    dst = page[with_tail].long()
    keep = torch.arange(pt, device=kv.device) < rest[with_tail][:, None]
    keep = keep[None, :, :, None, None] if s["case"]["layout"] == "token" else keep[None, :, None, :, None]
    kv[:, dst] = torch.where(keep, kv[:, src], kv[:, dst])


def _compact(s):
    b, pages, kv = _views(s["book"], *s["shape"]), s["shape"][2], s["kv"]
    used = b["refs"] > 0
    live = int(used.sum())
    hole = torch.nonzero(~used[:live]).flatten()
    move = torch.nonzero(used[live:]).flatten() + live
    kv[:, hole] = kv[:, move]
    to = torch.arange(pages, device=kv.device, dtype=torch.int32)
    to[move] = hole.to(torch.int32)
    held = torch.arange(s["shape"][1], device=kv.device) < ((b["lens"] + s["case"]["pt"] - 1) // s["case"]["pt"])[:, None]
    b["table"].copy_(torch.where(held, to[b["table"].long()], b["table"]))
    b["refs"][hole] = b["refs"][move]
    b["refs"][live:] = 0
    b["free"][:pages - live] = torch.arange(pages - 1, live - 1, -1, device=kv.device, dtype=torch.int32)
    b["counts"][0] = pages - live


def _resize(s):
    b, pt = _views(s["book"], *s["shape"]), s["case"]["pt"]
    q, to = s["seqs"].long(), s["to"]
    had, has = (b["lens"][q] + pt - 1) // pt, (to + pt - 1) // pt
    j = torch.arange(s["shape"][1], device=to.device)
    theirs = b["table"][q]
    before = b["refs"].clone()
    gone = (j >= has[:, None]) & (j < had[:, None])
    b["refs"].index_add_(0, theirs.flatten(), -gone.flatten().to(torch.int32))
    zero = torch.nonzero((before > 0) & (b["refs"] == 0)).flatten().flip(0).to(torch.int32)
    b["free"][b["counts"][0] + torch.arange(len(zero), device=to.device)] = zero
    top = b["counts"][0] + len(zero)
    need = (has - had).clamp(min=0)
    come = (j >= had[:, None]) & (j < has[:, None])
    k = (torch.cumsum(need, 0) - need)[:, None] + j - had[:, None]
    page = b["free"][torch.where(come, top - 1 - k, 0)]
    b["table"][q] = torch.where(come, page, theirs)
    b["refs"].index_add_(0, page.flatten(), come.flatten().to(torch.int32))
    b["lens"][q] = to
    b["counts"][0] = top - need.sum()


def _attention(s):
    c, b = s["case"], _views(s["book"], *s["shape"])
    kv = s["kv"] if c["layout"] == "token" else s["kv"].transpose(2, 3)
    bs, t, hk, d = s["k"].shape
    gr = c["groups"]
    q = s["q"].float().view(bs, t, hk, gr, d).permute(0, 2, 1, 3, 4).reshape(bs, hk, t * gr, d)
    seqs = s["seqs"].long()
    length = b["lens"][seqs]
    pages = b["table"][seqs][:, :-(-c["ctx"] // c["pt"])].long()
    k = kv[0][pages].reshape(bs, -1, hk, d).float().permute(0, 2, 3, 1).contiguous()
    far = torch.arange(k.shape[3], device=q.device) >= length[:, None]
    x = torch.matmul(q, k).masked_fill_(far[:, None, None], -math.inf)
    del k
    y = torch.matmul(q, s["k"].float().permute(0, 2, 3, 1).contiguous()).view(bs, hk, t, gr, t)
    i = torch.arange(t, device=q.device)
    if s["mask"] is None:
        sees = (i[None, :] <= i[:, None])[None].expand(bs, t, t)
    else:
        sees = ((s["mask"][:, :, i // 64] >> (i % 64)) & 1) > 0
    there = torch.ones(bs, t, dtype=torch.bool, device=q.device) if s["nodes"] is None else i < s["nodes"][:, None]
    sees = sees & there[:, None, :]
    y = y.masked_fill_(~sees[:, None, :, None, :], -math.inf).view(bs, hk, t * gr, t)
    x = torch.cat([x, y], 3).mul_(1 / math.sqrt(d))
    top = x.amax(3, keepdim=True)
    x = x.sub_(top.clamp(min=-3e38)).exp_()
    total = x.sum(3, keepdim=True)
    v = torch.cat([kv[1][pages].reshape(bs, -1, hk, d), s["v"]], 1).float().permute(0, 2, 1, 3).contiguous()
    o = torch.matmul(x, v) / total.clamp(min=1e-38)
    lse = top + total.log()
    o = o.view(bs, hk, t, gr, d).permute(0, 2, 1, 3, 4).reshape(bs, t, hk * gr, d)
    lse = lse.view(bs, hk, t, gr).permute(0, 2, 1, 3).reshape(bs, t, hk * gr)
    o = torch.where(there[:, :, None, None], o, 0.0)
    return {"out": o.to(s["q"].dtype), "lse": torch.where(there[:, :, None], lse, -math.inf)}


def work(case):
    c = case
    if c["op"] == "attention":
        keys = sum(_used(c)) + c["batch"] * c["nodes"]
        hq, rows = c["heads"] * c["groups"], c["batch"] * c["nodes"]
        return {"bytes": 2 * keys * _token(c) + 4 * rows * hq * c["dim"] + 4 * rows * hq, "flops": 4.0 * c["dim"] * hq * c["nodes"] * keys}
    if c["op"] == "copy":
        return {"bytes": 2 * c["n"] * c["pools"] * _page(c) + 8 * c["n"], "flops": 0}
    if c["op"] == "append":
        n = min(c["n"], sum(_used(c)))
        return {"bytes": 2 * (n - n // 8) * c["pools"] * _token(c) + 16 * n, "flops": 0}
    if c["op"] == "fork":
        rest, pages = sum(v % c["pt"] for v in _used(c)), _live(c)
        return {"bytes": c["ways"] * (2 * c["pools"] * rest * _token(c) + 16 * pages), "flops": 0}
    if c["op"] == "compact":
        return {"bytes": 2 * c["pools"] * _moved(c) * _page(c) + 4 * _live(c) + 8 * _moved(c) + 12 * _pages(c), "flops": 0}
    # a third ends, a third grows by a little, a third begins with half the longest prompt on average
    n, whole = c["listed"], sum(_npg(v, c["pt"]) for i, v in enumerate(_used(c)[:c["listed"]]) if i % 3 == 0)
    return {"bytes": 16 * (whole + n // 3 * _npg(c["ctx"], c["pt"]) // 2 + n), "flops": 0}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    rows, width, pages = s["shape"]
    if c["op"] == "attention":
        return _exact_attention(s)
    pt, kv = c["pt"], s["kv"]
    flat = s["held"].tolist()
    table = [flat[i * width:(i + 1) * width] for i in range(rows)]
    lens = flat[rows * width:rows * width + rows]
    refs = flat[rows * width + rows:rows * width + rows + pages]
    free = flat[rows * width + rows + pages:rows * width + rows + 2 * pages]
    top = flat[rows * width + rows + 2 * pages]
    moves = []  # (from page, to page, tokens)
    if c["op"] == "copy":
        moves = [(a, b, pt) for a, b in zip(s["src"].tolist(), s["dst"].tolist())]
    elif c["op"] == "append":
        for q, p, x in zip(s["seqs"].tolist(), s["at"].tolist(), s["index"].tolist()):
            if q >= 0:
                page, off = table[q][p // pt], p % pt
                if c["layout"] == "token":
                    kv[:, page, off] = s["new"][:, x]
                else:
                    kv[:, page, :, off] = s["new"][:, x]
        return {"kv": kv}
    elif c["op"] == "fork":
        for a, b in zip(s["parents"].tolist(), s["children"].tolist()):
            lens[b] = lens[a]
            for j in range(lens[a] // pt):
                table[b][j] = table[a][j]
                refs[table[a][j]] += 1
            if lens[a] % pt:
                top -= 1
                page = free[top]
                table[b][lens[a] // pt] = page
                refs[page] = 1
                moves.append((table[a][lens[a] // pt], page, lens[a] % pt))
    elif c["op"] == "compact":
        live = sum(r > 0 for r in refs)
        hole, name = 0, {}
        for p in range(live, pages):
            if refs[p]:
                while refs[hole]:
                    hole += 1
                moves.append((p, hole, pt))
                name[p], refs[hole], refs[p] = hole, refs[p], 0
        for q in range(rows):
            for j in range(_npg(lens[q], pt)):
                table[q][j] = name.get(table[q][j], table[q][j])
        top = pages - live
        free[:top] = range(pages - 1, live - 1, -1)
    else:
        freed = []
        todo = list(zip(s["seqs"].tolist(), s["to"].tolist()))
        for q, to in todo:
            for j in range(_npg(to, pt), _npg(lens[q], pt)):
                refs[table[q][j]] -= 1
                if not refs[table[q][j]]:
                    freed.append(table[q][j])
        for page in sorted(freed, reverse=True):
            free[top] = page
            top += 1
        for q, to in todo:
            for j in range(_npg(lens[q], pt), _npg(to, pt)):
                top -= 1
                table[q][j] = free[top]
                refs[free[top]] = 1
            lens[q] = to
    for a, b, n in moves:
        if c["layout"] == "token":
            kv[:, b, :n] = kv[:, a, :n]
        else:
            kv[:, b, :, :n] = kv[:, a, :, :n]
    if c["op"] == "copy":
        return {"kv": kv}
    book = torch.tensor([x for r in table for x in r] + lens + refs + free + [top, 0, 0, 0], dtype=torch.int32)
    return {"book": book} if c["op"] == "resize" else {"kv": kv, "book": book}


def _exact_attention(s):
    c, b = s["case"], _views(s["book"], *s["shape"])
    pt, gr, d, t = c["pt"], c["groups"], c["dim"], c["nodes"]
    dev, dtype = s["q"].device, torch.float64
    out = torch.zeros(s["q"].shape, dtype=dtype, device=dev)
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=dtype, device=dev)
    for i, q in enumerate(s["seqs"].tolist()):
        n = int(b["lens"][q])
        page = b["table"][q, :_npg(n, pt)].long()
        count = t if s["nodes"] is None else int(s["nodes"][i])
        words = None if s["mask"] is None else [[w & (2 ** 64 - 1) for w in r] for r in s["mask"][i].tolist()]
        sees = [[j <= r if words is None else bool(words[r][j // 64] >> (j % 64) & 1) for j in range(count)] for r in range(count)]
        sees = torch.tensor(sees, dtype=torch.bool, device=dev).view(count, count)
        for h in range(c["heads"]):
            pool = [s["kv"][z][page][:, :, h] if c["layout"] == "token" else s["kv"][z][page][:, h] for z in (0, 1)]
            key = torch.cat([pool[0].reshape(-1, d)[:n], s["k"][i, :count, h]]).to(dtype)
            val = torch.cat([pool[1].reshape(-1, d)[:n], s["v"][i, :count, h]]).to(dtype)
            x = s["q"][i, :count, h * gr:(h + 1) * gr].to(dtype).reshape(count * gr, d) @ key.T.contiguous() / math.sqrt(d)
            x[:, n:].masked_fill_(~sees.repeat_interleave(gr, 0), -math.inf)
            z = torch.logsumexp(x, 1)
            out[i, :count, h * gr:(h + 1) * gr] = (torch.exp(x - z[:, None]) @ val).view(count, gr, d)
            lse[i, :count, h * gr:(h + 1) * gr] = z.view(count, gr)
    return {"out": out, "lse": lse}
