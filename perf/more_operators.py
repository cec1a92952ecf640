"""Cases of the verification of drafted tokens, of attention over a window of a paged cache, and of a paged cache held in 4 bits.

Verification walks a tree of drafted tokens: node 0 holds; a child is accepted where its random number, times the probability that it was drafted with, is below
what the target's distribution has left for its token; what a rejected one was drafted from is taken off. The next token is drawn from what is left.
The cache and its bookkeeping are laid out as in operators.py: pools of pages, and one int32 tensor of table, lens, refs, free and counts.
In 4 bits a head is blocks of 32 elements: two signed numbers of {0, 0.5, 1, 1.5, 2, 3, 4, 6} a byte (the first one low), then a byte for each block, the power
of two (less 127) that all of it is multiplied by, and zeros up to a multiple of four bytes.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}

LISTED = [
    # a few chat requests, each with a short chain from a small draft model: a call whose cost is its launches
    {"name": "verify_chains_small", "op": "verify", "batch": 3, "nodes": 5, "kids": 1, "vocab": 32000, "draft": True, "ragged": False, "dtype": "fp32"},
    # a full batch of chains, large vocabulary: the rows that the next tokens are drawn from
    {"name": "verify_chains_64", "op": "verify", "batch": 64, "nodes": 8, "kids": 1, "vocab": 131072, "draft": True, "ragged": True, "dtype": "fp32"},
    # wide trees of the draft's best tokens, which are not drawn at random; odd vocabulary
    {"name": "verify_trees_best", "op": "verify", "batch": 16, "nodes": 64, "kids": 4, "vocab": 100003, "draft": False, "ragged": True, "dtype": "bf16"},
    # small trees whose branches are drawn from the draft's probabilities
    {"name": "verify_trees_drawn", "op": "verify", "batch": 8, "nodes": 13, "kids": 3, "vocab": 50001, "draft": True, "ragged": False, "dtype": "fp32"},
    # single tokens of a few sequences that see little more than the last hundred
    {"name": "window_short", "op": "attention", "bits": 16, "batch": 4, "nodes": 1, "tree": False, "ctx": 700, "window": 128, "sinks": 4, "groups": 4, "pt": 16, "heads": 2,
     "dim": 64, "layout": "head", "dtype": "fp16"},
    # single tokens of a ragged batch of long sequences
    {"name": "window_decode_64", "op": "attention", "bits": 16, "batch": 64, "nodes": 1, "tree": False, "ctx": 32767, "window": 4096, "sinks": 4, "groups": 4, "pt": 16, "heads": 8,
     "dim": 128, "layout": "token", "dtype": "bf16"},
    # wide trees, whose nodes' windows begin at different tokens
    {"name": "window_trees_64", "op": "attention", "bits": 16, "batch": 16, "nodes": 64, "tree": True, "ctx": 16383, "window": 2000, "sinks": 16, "groups": 4, "pt": 32, "heads": 8,
     "dim": 128, "layout": "token", "dtype": "bf16"},
    # accepted tokens of a few sequences rounded into a small cache and read back
    {"name": "fp4_append_small", "op": "append", "n": 13, "seqs": 5, "ctx": 90, "pools": 4, "pt": 16, "heads": 3, "dim": 64, "layout": "head", "dtype": "fp16"},
    # a prompt rounded into the pools of 32 layers and read back
    {"name": "fp4_append_prompt", "op": "append", "n": 4000, "seqs": 2, "ctx": 4001, "pools": 64, "pt": 32, "heads": 8, "dim": 128, "layout": "head", "dtype": "bf16"},
    # single tokens of a few short sequences
    {"name": "fp4_short", "op": "attention", "bits": 4, "batch": 4, "nodes": 1, "tree": False, "ctx": 333, "window": 0, "sinks": 0, "groups": 4, "pt": 16, "heads": 2,
     "dim": 64, "layout": "head", "dtype": "fp16"},
    # single tokens of a large ragged batch: the cache's bytes decide
    {"name": "fp4_decode_64", "op": "attention", "bits": 4, "batch": 64, "nodes": 1, "tree": False, "ctx": 8191, "window": 0, "sinks": 0, "groups": 4, "pt": 16, "heads": 8,
     "dim": 128, "layout": "head", "dtype": "bf16"},
    # wide trees over long contexts: products count more than bytes
    {"name": "fp4_trees_64", "op": "attention", "bits": 4, "batch": 16, "nodes": 64, "tree": True, "ctx": 16383, "window": 0, "sinks": 0, "groups": 4, "pt": 32, "heads": 8,
     "dim": 128, "layout": "token", "dtype": "bf16"},
]


def listed():
    return [dict(c) for c in LISTED]


def _log(rng, a, b):
    return min(b, max(a, int(round(math.exp(rng.uniform(math.log(a), math.log(b + 0.49)))))))


def draw(rng):
    op = rng.choice(["verify", "verify", "attention", "attention", "attention", "append"])
    if op == "verify":
        while True:
            c = {"op": op, "batch": _log(rng, 1, 64), "nodes": _log(rng, 1, 100), "kids": rng.choice([1, 1, 2, 3, 5]), "vocab": _log(rng, 500, 131072), "draft": rng.random() < 0.6,
                 "ragged": rng.random() < 0.5, "dtype": rng.choice(["fp32", "fp32", "bf16", "fp16"])}
            if c["batch"] * c["nodes"] * c["vocab"] <= 1 << 26:
                return c
    c = {"op": op, "layout": rng.choice(["token", "head"]), "dtype": rng.choice(["bf16", "fp16"]), "pt": rng.choice([1, 5, 8, 16, 16, 20, 32, 64]),
         "heads": rng.choice([1, 2, 3, 4, 8]), "dim": rng.choice([64, 96, 128, 128, 256])}
    if op == "append":
        while True:
            c.update(n=_log(rng, 1, 4000), seqs=_log(rng, 1, 100), ctx=_log(rng, 1, 2000), pools=2 * _log(rng, 1, 32))
            if c["pools"] * _pages(c) * c["pt"] * c["heads"] * c["dim"] <= 1 << 31:
                return c
    while True:
        c.update(bits=rng.choice([4, 4, 16]), batch=_log(rng, 1, 64), nodes=rng.choice([1, 1, _log(rng, 2, 100), _log(rng, 2, 100)]), ctx=_log(rng, 1, 20000),
                 groups=rng.choice([1, 2, 4, 5, 7, 8, 16]), window=0, sinks=0, tree=rng.random() < 0.7)
        if c["bits"] == 16 or rng.random() < 0.5:
            c.update(window=_log(rng, 1, 4096), sinks=rng.choice([0, 1, 4, rng.randrange(100)]))
        c["tree"] = c["tree"] and c["nodes"] > 1
        keys = c["batch"] * c["heads"] * c["dim"] * (c["ctx"] + c["nodes"])
        if keys <= 16 * 8 * 128 * 16384 and keys * c["nodes"] * c["groups"] <= 16 * 8 * 128 * 16384 * 256:
            return c


def _lens(n, ctx):
    return [max(1, (i + 1) * ctx // n) for i in range(n)]


def _npg(length, pt):
    return -(-length // pt)


def _pages(c):
    return sum(_npg(v, c["pt"]) for v in _lens(c.get("batch") or c["seqs"], c["ctx"])) + 3


def _head_bytes(dim):
    return dim // 2 + (dim // 32 + 3) // 4 * 4


def _limits(dtype):
    """Smallest and largest power of two of a block, so that all it stands for are numbers of the type."""
    return (-23, 13) if dtype == torch.float16 else (-126, 125)


def _rounded(x):
    """x [..., dim] in 4 bits: uint8 [..., head bytes]."""
    dim, (low, high) = x.shape[-1], _limits(x.dtype)
    y = x.float().unflatten(-1, (dim // 32, 32))
    top = y.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top)
    e = (e - 3 + (m >= 0.875).to(e.dtype)).clamp(low, high)
    y = torch.ldexp(y, -e)
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5) + 8 * torch.signbit(y).to(torch.uint8)).flatten(-2)
    parts = [code[..., 0::2] | code[..., 1::2] << 4, (e + 127).to(torch.uint8).squeeze(-1)]
    pad = _head_bytes(dim) - dim // 2 - dim // 32
    return torch.cat(parts + [torch.zeros(x.shape[:-1] + (pad,), dtype=torch.uint8, device=x.device)], -1)


def _numbers(b, dim):
    """What uint8 [..., head bytes] stands for, in 32 bits [..., dim]."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=b.device)
    code = torch.stack([b[..., :dim // 2] & 15, b[..., :dim // 2] >> 4], -1).flatten(-2)
    e = b[..., dim // 2:dim // 2 + dim // 32].to(torch.int32) - 127
    return torch.ldexp(table[code.int()].unflatten(-1, (dim // 32, 32)), e[..., None]).flatten(-2)


def _views(book, rows, width):
    a = rows * width
    return {"table": book[:a].view(rows, width), "lens": book[a:a + rows]}


def _filled(shape, dtype, g, dev):
    return torch.empty(shape, dtype=dtype, device=dev).normal_(generator=g)


def prepare(case, seed):
    c, dev = case, torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    h = torch.Generator().manual_seed(seed)

    def ints(v):
        return torch.as_tensor(v, dtype=torch.int32).to(dev)

    if c["op"] == "verify":
        return _prepare_verify(c, g, h, ints, dev)
    pt, pages, dtype, dim = c["pt"], _pages(c), DTYPES[c["dtype"]], c["dim"]
    rows = c.get("batch") or c["seqs"]
    lens = torch.tensor(_lens(rows, c["ctx"]))[torch.randperm(rows, generator=h)]
    width = _npg(c["ctx"], pt) + 1
    pools = c.get("pools", 2)
    bits = c.get("bits", 4)
    page = (pt, c["heads"]) if c["layout"] == "token" else (c["heads"], pt)
    if bits == 16:
        kv = _filled((pools, pages) + page + (dim,), dtype, g, dev)
    else:
        kv = torch.empty((pools, pages) + page + (_head_bytes(dim),), dtype=torch.uint8, device=dev)
        step = max(1, (1 << 26) // (pt * c["heads"] * dim))
        for p in range(pools if c["op"] == "attention" else 1):  # what append does not write is alike in all pools
            for i in range(0, pages, step):
                kv[p, i:i + step] = _rounded(_filled((min(step, pages - i),) + page + (dim,), dtype, g, dev))
        if c["op"] == "append":
            kv[1:] = kv[0]
    # pages at random places of the cache
    n = _npg(lens, pt)
    table = torch.zeros(rows, width, dtype=torch.int64)
    at = torch.randperm(pages, generator=h)[:int(n.sum())]
    table[torch.arange(width) < n[:, None]] = at
    refs = torch.zeros(pages, dtype=torch.int64)
    refs[at] = 1
    empty = torch.nonzero(refs == 0).flatten()
    free = torch.zeros(pages, dtype=torch.int64)
    free[:len(empty)] = empty
    book = ints(torch.cat([table.flatten(), lens, refs, free, torch.tensor([len(empty), 0, 0, 0])]))
    s = {"case": c, "kv": kv, "book": book, "shape": (rows, width, pages)}
    if c["op"] == "append":
        # tokens of the sequences, out of order, a few of those that a model's pass gave rows for; one in eight is padding
        tok = torch.cat([torch.stack([torch.full((int(v),), i), torch.arange(int(v))], 1) for i, v in enumerate(lens)])
        tok = tok[torch.randperm(len(tok), generator=h)[:c["n"]]]
        seqs = tok[:, 0].clone()
        seqs[7::8] = -1
        given = len(tok) + 1 + len(tok) // 8
        s.update(seqs=ints(seqs), at=ints(tok[:, 1]), index=ints(torch.randperm(given, generator=h)[:len(tok)]), new=_filled((pools, given, c["heads"], dim), dtype, g, dev))
    else:
        b, t, hk, hq = c["batch"], c["nodes"], c["heads"], c["heads"] * c["groups"]
        s.update(q=_filled((b, t, hq, dim), dtype, g, dev), k=_filled((b, t, hk, dim), dtype, g, dev), v=_filled((b, t, hk, dim), dtype, g, dev),
                 seqs=ints(torch.randperm(rows, generator=h)), mask=None, nodes=None, depths=None)
        if c["tree"]:
            parent = (torch.rand(b, t, generator=h) * torch.arange(t)).long()
            sees, depth = _tree(parent)
            s["mask"] = _words(sees).to(dev)
            s["depths"] = ints(depth)
            s["nodes"] = ints([t - t // 3 if i % 3 == 2 else t for i in range(b)])
    if own:  # the handle that a server keeps
        from copy_reduce_amd.torch_api import PagedCache, tree_attention_workspace
        s["cache"] = PagedCache(kv, page_tokens=pt, max_seqs=rows, max_pages=width, layout=c["layout"], state=book, fp4=dtype if bits == 4 else None)
        if c["op"] == "attention":
            s["workspace"] = tree_attention_workspace(s["q"], s["cache"])
    return s


def _tree(parent):
    """(which nodes each sees: itself and its ancestors, depths) of trees whose nodes follow their parents."""
    b, t = parent.shape
    sees = torch.zeros(b, t, t, dtype=torch.bool)
    sees[:, 0, 0] = True
    for i in range(1, t):
        sees[:, i] = sees[torch.arange(b), parent[:, i]]
        sees[:, i, i] = True
    return sees, sees.sum(2) - 1


def _words(sees):
    b, t, _ = sees.shape
    words = -(-t // 64)
    bits = torch.zeros(b, t, words * 64, dtype=torch.int64)
    bits[..., :t] = sees
    return (bits.view(b, t, words, 64) * (torch.ones((), dtype=torch.int64) << torch.arange(64))).sum(-1)


def _prepare_verify(c, g, h, ints, dev):
    b, t, v, dtype = c["batch"], c["nodes"], c["vocab"], DTYPES[c["dtype"]]
    # a draft that mostly agrees with the target: its logits are the target's with some noise
    probs, drafts = torch.empty(b, t, v, dtype=dtype, device=dev), torch.empty(b, t, v, dtype=dtype, device=dev)
    for i in range(b):
        x = 3 * _filled((t, v), torch.float32, g, dev)
        probs[i] = torch.softmax(x, 1)
        drafts[i] = torch.softmax(x + 0.5 * _filled((t, v), torch.float32, g, dev), 1)
    # node i's parent is the first that has fewer than its share of children, now and then one before
    parent = torch.zeros(b, t, dtype=torch.int64)
    for i in range(1, t):
        parent[:, i] = torch.clamp((i - 1) // c["kids"] - (torch.rand(b, generator=h) < 0.2 * (c["kids"] > 1)).long(), min=0)
    rank = ((parent[:, None, :] == parent[:, :, None]) & (torch.arange(t)[None, None, :] < torch.arange(t)[None, :, None])
            & (torch.arange(t) > 0)).sum(2)  # place among the children of its parent
    par, rank = parent.to(dev), rank.to(dev)
    most = int(rank.max()) + 1
    rows = drafts.view(b * t, v)
    if c["draft"]:
        got = torch.multinomial(rows.float(), most, replacement=True, generator=g)
    else:
        got = torch.topk(rows.float(), min(most, v), dim=1).indices
    tokens = got.view(b, t, -1)[torch.arange(b, device=dev)[:, None], par, rank.clamp(max=got.shape[1] - 1)].to(torch.int32)
    nodes = ints([t - t // 3 if c["ragged"] and i % 3 == 2 else t for i in range(b)])
    rows = b + 3
    pt, width = 16, 40
    lens = torch.randint(0, 500, (rows,), generator=h)
    book = ints(torch.cat([torch.zeros(rows * width, dtype=torch.int64), lens, torch.zeros(2 * rows * width + 4, dtype=torch.int64)]))
    s = {"case": c, "probs": probs, "drafts": drafts if c["draft"] else None, "tokens": tokens, "parents": None if c["kids"] == 1 else par.to(torch.int32),
         "uniform": torch.rand(b, t, device=dev, generator=g), "nodes": nodes, "seqs": ints(torch.randperm(rows, generator=h)[:b]), "book": book, "shape": (rows, width, rows * width),
         "sees": None if c["kids"] == 1 else _tree(parent)[0].to(dev)}
    if own:  # the cache whose sequences the accepted tokens go to
        from copy_reduce_amd.torch_api import PagedCache, verify_drafts_workspace
        s["kv"] = torch.empty(2, rows * width, pt, 1, 8, dtype=torch.bfloat16, device=dev)
        s["cache"] = PagedCache(s["kv"], page_tokens=pt, max_seqs=rows, max_pages=width, state=book)
        s["workspace"] = verify_drafts_workspace(probs)
    return s


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        from copy_reduce_amd.torch_api import tree_attention, verify_drafts
        if op == "verify":
            r = verify_drafts(s["probs"], s["tokens"], s["uniform"], parents=s["parents"], draft_probs=s["drafts"], nodes=s["nodes"], cache=s["cache"], seqs=s["seqs"],
                              workspace=s["workspace"])
            return {"count": r.count, "path": r.path, "token": r.token, "lens": r.lens, "rows": r.append_seqs, "positions": r.append_positions, "index": r.append_index}
        if op == "append":
            s["cache"].append(s["new"], s["seqs"], s["at"], index=s["index"])
            return {"values": s["cache"].read(s["seqs"], s["at"])}
        out, lse = tree_attention(s["q"], s["k"], s["v"], s["cache"], 0, s["seqs"], mask=s["mask"], nodes=s["nodes"], window=s["case"]["window"] or None,
                                  sinks=s["case"]["sinks"], depths=s["depths"], workspace=s["workspace"])
        return {"out": out, "lse": lse}
    return {"verify": _verify, "append": _append, "attention": _attention}[op](s)


def _verify(s):
    p, q, x, u = s["probs"], s["drafts"], s["tokens"].long(), s["uniform"].double()
    b, t, v = p.shape
    dev = p.device
    i, at = torch.arange(t, device=dev), torch.arange(b, device=dev)[:, None]
    par = (i - 1).clamp(min=0).expand(b, t) if s["parents"] is None else s["parents"].long()
    there = i < s["nodes"][:, None]
    px = p[at, par, x].double()
    if s["parents"] is None:  # chains
        ok = there & (i > 0) & (u * (1.0 if q is None else q[at, par, x].double()) < px)
        ok[:, 0] = there[:, 0]
        on = torch.cumprod(ok.int(), 1) > 0
    else:
        brother = (par[:, :, None] == par[:, None, :]) & (i[:, None] > i) & (i > 0)
        if q is None:
            again = (brother & (x[:, :, None] == x[:, None, :])).any(2)
            px = torch.where(again, 0.0, px)
            left = 1.0 - (brother * px[:, None, :]).sum(2)
            ok = u * left < px
        else:  # what is left of a distribution after each of its children in turn
            rank = brother.sum(2)
            qx = q[at, par, x].double()
            ok = u * qx < px
            r = p.double()
            for k in range(1, 2 * s["case"]["kids"]):
                r = (r - q).clamp_(min=0)
                r /= r.sum(2, keepdim=True).clamp_(min=1e-300)
                ok = torch.where(rank == k, u * qx < r[at, par, x], ok)
        ok = ok & there & (i > 0)
        first = ok & ~(brother & ok[:, None, :]).any(2)
        first[:, 0] = there[:, 0]
        on = (first[:, None, :] | ~s["sees"]).all(2) & there
    count = on.sum(1)
    cur = torch.where(on, i, 0).amax(1)
    row, below = p[at[:, 0], cur].double(), there & (par == cur[:, None]) & (i > 0)
    if q is None:
        tried = torch.zeros(b, v, dtype=torch.int32, device=dev).scatter_add_(1, x, below.to(torch.int32))
        left = torch.where(tried > 0, 0.0, row)
    else:
        left, d, tried = row, q[at[:, 0], cur].double(), below.sum(1, keepdim=True)
        for k in range(2 * s["case"]["kids"] if s["case"]["kids"] > 1 else 1):
            rest = (left - d).clamp_(min=0)
            left = torch.where(tried > k, rest / rest.sum(1, keepdim=True).clamp_(min=1e-300), left)
    left = torch.where(left.sum(1, keepdim=True) > 0, left, row)
    mass = torch.cumsum(left, 1)
    token = torch.searchsorted(mass, u[:, :1] * mass[:, -1:], right=True).squeeze(1).to(torch.int32)
    token = torch.where(there[:, 0], token, -1)
    place = torch.cumsum(on, 1) - 1
    path = torch.full((b, t + 1), -1, dtype=torch.int32, device=dev)
    path.scatter_(1, torch.where(on, place, t), i.to(torch.int32).expand(b, t))
    path = path[:, :t]
    had = _views(s["book"], *s["shape"][:2])["lens"][s["seqs"].long()]
    real = path >= 0
    return {"count": count.to(torch.int32), "path": path, "token": token, "lens": (had + count).to(torch.int32), "rows": torch.where(real, s["seqs"][:, None], -1).flatten(),
            "positions": torch.where(real, had[:, None] + i, 0).to(torch.int32).flatten(), "index": torch.where(real, at * t + path, 0).to(torch.int32).flatten()}


def _append(s):
    b, c = _views(s["book"], *s["shape"][:2]), s["case"]
    there = s["seqs"] >= 0
    q, at, x = s["seqs"].clamp(min=0).long(), s["at"].long(), s["index"].long()
    page, off = b["table"][q, at // c["pt"]].long(), at % c["pt"]
    by_token = s["kv"] if c["layout"] == "token" else s["kv"].transpose(2, 3)
    by_token[:, page[there], off[there]] = _rounded(s["new"][:, x[there]])
    return {"values": (_numbers(by_token[:, page, off], c["dim"]) * there[:, None, None]).to(s["new"].dtype)}


def _attention(s):
    c, b = s["case"], _views(s["book"], *s["shape"][:2])
    kv = s["kv"] if c["layout"] == "token" else s["kv"].transpose(2, 3)
    bs, t, hk, d = s["k"].shape
    gr, w = c["groups"], c["window"]
    dev = s["q"].device
    i = torch.arange(t, device=dev)
    depth = i.expand(bs, t) if s["depths"] is None else s["depths"]
    q = s["q"].float().view(bs, t, hk, gr, d).permute(0, 2, 1, 3, 4).reshape(bs, hk, t * gr, d)
    seqs = s["seqs"].long()
    length = b["lens"][seqs][:, None]
    if w and w + c["sinks"] < c["ctx"]:  # only the tokens that some node sees
        j = torch.arange(c["sinks"] + w - 1, device=dev)
        at = torch.where(j < c["sinks"], j, j - c["sinks"] + (length + 1 - w).clamp(min=c["sinks"]))
    else:
        at = torch.arange(c["ctx"], device=dev).expand(bs, -1)
    page, off = b["table"][seqs[:, None], (at // c["pt"]).clamp(max=s["shape"][1] - 1).long()].long(), at % c["pt"]

    def held(z):
        x = kv[z][page, off]
        return (x if c["bits"] == 16 else _numbers(x, d)).float()

    far = (at >= length)[:, None, :]
    if w:
        far = far | ((at[:, None, :] >= c["sinks"]) & (at[:, None, :] <= (length + depth - w)[:, :, None]))
    x = torch.matmul(q, held(0).permute(0, 2, 3, 1).contiguous())
    x = x.view(bs, hk, t, gr, -1).masked_fill_(far[:, None, :, None, :], -math.inf).view(bs, hk, t * gr, -1)
    y = torch.matmul(q, s["k"].float().permute(0, 2, 3, 1).contiguous()).view(bs, hk, t, gr, t)
    if s["mask"] is None:
        sees = (i[None, :] <= i[:, None])[None].expand(bs, t, t)
    else:
        sees = ((s["mask"][:, :, i // 64] >> (i % 64)) & 1) > 0
    if w:
        sees = sees & (((length + depth) < c["sinks"])[:, None, :] | (depth[:, :, None] - depth[:, None, :] < w))
    there = torch.ones(bs, t, dtype=torch.bool, device=dev) if s["nodes"] is None else i < s["nodes"][:, None]
    sees = sees & there[:, None, :]
    y = y.masked_fill_(~sees[:, None, :, None, :], -math.inf).view(bs, hk, t * gr, t)
    x = torch.cat([x, y], 3).mul_(1 / math.sqrt(d))
    top = x.amax(3, keepdim=True)
    x = x.sub_(top.clamp(min=-3e38)).exp_()
    total = x.sum(3, keepdim=True)
    v = torch.cat([held(1), s["v"].float()], 1).permute(0, 2, 1, 3).contiguous()
    o = torch.matmul(x, v) / total.clamp(min=1e-38)
    lse = top + total.log()
    o = o.view(bs, hk, t, gr, d).permute(0, 2, 1, 3, 4).reshape(bs, t, hk * gr, d)
    lse = lse.view(bs, hk, t, gr).permute(0, 2, 1, 3).reshape(bs, t, hk * gr)
    o = torch.where(there[:, :, None, None], o, 0.0)
    return {"out": o.to(s["q"].dtype), "lse": torch.where(there[:, :, None], lse, -math.inf)}


def work(case):
    c = case
    if c["op"] == "verify":  # a row of each distribution for each sequence, and a few numbers for each node
        size = DTYPES[c["dtype"]].itemsize
        rows = 2 if c["draft"] else 1
        return {"bytes": c["batch"] * (rows * size * c["vocab"] + c["nodes"] * (24 + rows * size)), "flops": 0}
    token = 2 * c["heads"] * c["dim"]
    held = token if c.get("bits", 4) == 16 else c["heads"] * _head_bytes(c["dim"])
    if c["op"] == "append":
        n = min(c["n"], sum(_lens(c["seqs"], c["ctx"])))
        real = n - n // 8
        return {"bytes": c["pools"] * (real * (token + 2 * held) + n * token) + 16 * n, "flops": 0}
    lens = _lens(c["batch"], c["ctx"])
    if c["window"]:
        lens = [min(v, c["sinks"] + c["window"] - 1) for v in lens]
    rows, hq = c["batch"] * c["nodes"], c["heads"] * c["groups"]
    return {"bytes": 2 * sum(lens) * held + 2 * rows * token + 4 * rows * hq * c["dim"] + 4 * rows * hq, "flops": 4.0 * c["dim"] * hq * c["nodes"] * (sum(lens) + rows)}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "attention":
        return _exact_attention(s)
    if c["op"] == "append":
        return {"values": _exact_values(s)}
    return _exact_verify(s)


def _exact_verify(s):
    c = s["case"]
    b, t = c["batch"], c["nodes"]
    lens = _views(s["book"], *s["shape"][:2])["lens"].tolist()
    tokens, uniform, nodes, seqs = s["tokens"].tolist(), s["uniform"].tolist(), s["nodes"].tolist(), s["seqs"].tolist()
    parents = [[i - 1 for i in range(t)]] * b if s["parents"] is None else s["parents"].tolist()
    out = {k: [] for k in ("count", "path", "token", "lens", "rows", "positions", "index")}
    for i in range(b):
        path, token = [], -1
        if nodes[i] > 0:
            path = [0]
            left = s["probs"][i, 0].double()
            z = 1.0
            for n in range(1, nodes[i]):
                if parents[i][n] != path[-1]:
                    continue
                x = tokens[i][n]
                drafted = 1.0 if s["drafts"] is None else float(s["drafts"][i, path[-1], x].double())
                if uniform[i][n] * drafted * z < float(left[x]):
                    path.append(n)
                    left, z = s["probs"][i, n].double(), 1.0
                elif s["drafts"] is None:
                    z -= float(left[x])
                    left[x] = 0
                else:
                    left = torch.relu(left - s["drafts"][i, path[-1]].double() * z)
                    z = float(left.sum())
            if not bool(left.any()):
                left = s["probs"][i, path[-1]].double()
            mass = left.cumsum(0)
            token = int((mass <= uniform[i][0] * mass[-1]).sum())
        pad = t - len(path)
        at = lens[seqs[i]]
        out["count"].append(len(path))
        out["path"].append(path + [-1] * pad)
        out["token"].append(token)
        out["lens"].append(at + len(path))
        out["rows"] += [seqs[i]] * len(path) + [-1] * pad
        out["positions"] += [at + k for k in range(len(path))] + [0] * pad
        out["index"] += [i * t + n for n in path] + [0] * pad
    return {k: torch.tensor(v, dtype=torch.int32) for k, v in out.items()}


def _exact_values(s):
    """The nearest of the numbers that a block can hold, the one with an even code of two; written apart from _rounded()."""
    low, high = _limits(s["new"].dtype)
    steps = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=s["new"].device)
    out = torch.zeros((s["new"].shape[0], len(s["seqs"])) + s["new"].shape[2:], dtype=torch.float64, device=s["new"].device)
    real = torch.nonzero(s["seqs"] >= 0).flatten()
    for p in range(out.shape[0]):
        x = s["new"][p][s["index"].long()[real]].double()
        y = x.view(*x.shape[:-1], -1, 32)
        big = y.abs().amax(-1, keepdim=True)
        e = torch.floor(torch.log2(big.clamp(min=1e-300) / 7)) + 1
        e = torch.where(big < 7 * torch.exp2(e - 1), e - 1, torch.where(big >= 7 * torch.exp2(e), e + 1, e)).clamp(low, high)
        a = (y / torch.exp2(e)).abs()
        up = torch.searchsorted(steps, a.clamp(max=6)).clamp(1, 7)
        below, above = steps[up - 1], steps[up]
        nearer = torch.where(a - below < above - a, below, torch.where(a - below > above - a, above, torch.where(up % 2 == 0, above, below)))
        out[p, real] = (torch.where(y < 0, -nearer, nearer) * torch.exp2(e)).view(x.shape)
    return out


def _exact_attention(s):
    c, b = s["case"], _views(s["book"], *s["shape"][:2])
    pt, gr, d, t = c["pt"], c["groups"], c["dim"], c["nodes"]
    dev, dtype = s["q"].device, torch.float64
    out = torch.zeros(s["q"].shape, dtype=dtype, device=dev)
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=dtype, device=dev)
    signs = torch.tensor([1.0] * 8 + [-1.0] * 8, dtype=dtype, device=dev)
    sizes = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6] * 2, dtype=dtype, device=dev) * signs
    for i, q in enumerate(s["seqs"].tolist()):
        n = int(b["lens"][q])
        count = t if s["nodes"] is None else int(s["nodes"][i])
        words = None if s["mask"] is None else [[w & (2 ** 64 - 1) for w in r] for r in s["mask"][i].tolist()]
        depth = list(range(t)) if s["depths"] is None else s["depths"][i].tolist()
        at = list(range(n))
        if c["window"]:
            at = [j for j in at if j < c["sinks"] or n - j < c["window"]]
        place = torch.tensor(at, dtype=torch.int64, device=dev)
        sees = torch.ones(count, len(at) + count, dtype=torch.bool, device=dev)
        if c["window"]:
            away = n + torch.tensor(depth[:count], device=dev)[:, None] - place
            sees[:, :len(at)] = (place < c["sinks"]) | (away < c["window"])
        own_nodes = [[(j <= r if words is None else bool(words[r][j // 64] >> (j % 64) & 1))
                      and (not c["window"] or n + depth[j] < c["sinks"] or depth[r] - depth[j] < c["window"]) for j in range(count)] for r in range(count)]
        sees[:, len(at):] = torch.tensor(own_nodes, dtype=torch.bool, device=dev).view(count, count)
        page = b["table"][q].long()[place // pt]
        for h in range(c["heads"]):
            pool = [s["kv"][z][page, place % pt, h] if c["layout"] == "token" else s["kv"][z][page, h, place % pt] for z in (0, 1)]
            if c["bits"] == 4:
                for z in (0, 1):
                    raw = pool[z].long()
                    code = torch.empty(len(at), d, dtype=torch.int64, device=dev)
                    code[:, 0::2], code[:, 1::2] = raw[:, :d // 2] % 16, raw[:, :d // 2] // 16
                    pool[z] = sizes[code] * torch.exp2(raw[:, d // 2:d // 2 + d // 32].to(dtype) - 127).repeat_interleave(32, 1)
            key = torch.cat([pool[0].to(dtype), s["k"][i, :count, h].to(dtype)])
            val = torch.cat([pool[1].to(dtype), s["v"][i, :count, h].to(dtype)])
            x = s["q"][i, :count, h * gr:(h + 1) * gr].to(dtype).reshape(count * gr, d) @ key.T.contiguous() / math.sqrt(d)
            x.masked_fill_(~sees.repeat_interleave(gr, 0), -math.inf)
            z = torch.logsumexp(x, 1)
            out[i, :count, h * gr:(h + 1) * gr] = (torch.exp(x - z[:, None]) @ val).view(count, gr, d)
            lse[i, :count, h * gr:(h + 1) * gr] = z.view(count, gr)
    return {"out": out, "lse": lse}
