"""Plain models of what include/tb_serve.h promises, in 64 bits or in whole numbers, for the tests."""
import math

import torch

STEPS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
LIMITS = {torch.float16: (-23, 13), torch.bfloat16: (-126, 125)}


def head_bytes(dim):
    return dim // 2 + (dim // 32 + 3) // 4 * 4


def encode(x):
    """x [..., dim] of 16 bits -> uint8 [..., head_bytes(dim)]: the smallest power with max < 7 * 2^e, the nearest of the
    eight steps by distance, of two the even code."""
    dim, (low, high) = x.shape[-1], LIMITS[x.dtype]
    y = x.reshape(-1, dim // 32, 32).double()
    wild = ~torch.isfinite(y).all(2)
    y = torch.where(wild[:, :, None], 0.0, y)
    top = y.abs().amax(2)
    e = torch.full(top.shape, low)
    for _ in range(low, high):
        e += (top >= 7 * torch.exp2(e.double())) & (e < high)
    a = y.abs() / torch.exp2(e.double())[:, :, None]
    off = (a[..., None] - torch.tensor(STEPS, dtype=torch.float64)).abs()
    near = off == off.amin(3, keepdim=True)
    best = torch.where(near & (torch.arange(8) % 2 == 0), 2, near.int()).argmax(3)   # the even one of two
    code = (best + 8 * torch.signbit(y)).flatten(1).to(torch.uint8)
    code = torch.where(wild.repeat_interleave(32, 1), 0, code)
    powers = torch.where(wild, 255, e + 127).to(torch.uint8)
    pad = torch.zeros(len(code), head_bytes(dim) - dim // 2 - dim // 32, dtype=torch.uint8)
    return torch.cat([code[:, 0::2] | code[:, 1::2] << 4, powers, pad], 1).view(*x.shape[:-1], -1)


def decode(raw, dim):
    """What the bytes stand for, float64 [..., dim]."""
    flat = raw.reshape(-1, raw.shape[-1]).long()
    code = torch.stack([flat[:, :dim // 2] & 15, flat[:, :dim // 2] >> 4], 2).view(len(flat), dim)
    value = torch.tensor(STEPS + [-v for v in STEPS], dtype=torch.float64)[code]
    power = flat[:, dim // 2:dim // 2 + dim // 32]
    scale = torch.where(power == 255, math.nan, torch.exp2(power.double() - 127))
    return (value.view(len(flat), -1, 32) * scale[:, :, None]).view(*raw.shape[:-1], dim)


def window_attention(model, layer, q, k, v, seqs, mask=None, nodes=None, scale=None, window=None, sinks=0, depths=None):
    """As cache_model.attention, with a window: (out, lse, A, S, V)."""
    b, t, hq, d = q.shape
    hk = k.shape[2]
    g = hq // hk
    scale = 1 / math.sqrt(d) if scale is None else scale
    out = torch.zeros(b, t, hq, d, dtype=torch.float64)
    lse = torch.full((b, t, hq), -math.inf, dtype=torch.float64)
    a, s, big = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(lse)
    for i in range(b):
        row = int(seqs[i])
        if not 0 <= row < model.S:
            continue
        count = t if nodes is None else min(max(int(nodes[i]), 0), t)
        n = model.lens[row]
        depth = [u if depths is None else min(max(int(depths[i, u]), 0), count - 1) for u in range(count)]
        for x in range(count):
            at = [j for j in range(n) if window is None or j < sinks or n + depth[x] - j < window]
            sees = [u for u in range(count) if (u <= x if mask is None else int(mask[i, x, u // 64]) >> (u % 64) & 1)]
            if window is not None:
                sees = [u for u in sees if n + depth[u] < sinks or depth[x] - depth[u] < window]
            if not at and not sees:
                continue
            for h in range(hk):
                key = torch.cat([model.context(2 * layer, row, h)[at], k[i, sees, h].double()])
                val = torch.cat([model.context(2 * layer + 1, row, h)[at], v[i, sees, h].double()])
                qq = q[i, x, h * g:(h + 1) * g].double()
                y = qq @ key.T * scale
                z = torch.logsumexp(y, 1)
                w = torch.exp(y - z[:, None])
                out[i, x, h * g:(h + 1) * g] = w @ val
                lse[i, x, h * g:(h + 1) * g] = z
                a[i, x, h * g:(h + 1) * g] = w @ val.abs()
                s[i, x, h * g:(h + 1) * g] = (qq.abs() @ key.abs().T * abs(scale)).amax(1)
                big[i, x, h * g:(h + 1) * g] = val.abs().max()
    return out, lse, a, s, big


def verify(probs, tokens, uniform, parents=None, draft=None, nodes=None):
    """(count, path, token) of each sequence, the walk as the header tells it."""
    b, t, vocab = probs.shape
    found = []
    for i in range(b):
        n = t if nodes is None else min(max(int(nodes[i]), 0), t)
        if n == 0:
            found.append((0, [], -1))
            continue
        path, w, z = [0], probs[i, 0].double().clone(), 1.0
        for u in range(1, n):
            parent = u - 1 if parents is None else int(parents[i, u])
            x = int(tokens[i, u])
            if not 0 <= parent < u or parent != path[-1] or not 0 <= x < vocab:
                continue
            d = 1.0 if draft is None else float(draft[i, parent, x].double())
            if float(uniform[i, u].double()) * d * z < float(w[x]):
                path.append(u)
                w, z = probs[i, u].double().clone(), 1.0
            elif draft is None:
                z -= float(w[x])
                w[x] = 0
            else:
                w = (w - z * draft[i, parent].double()).clamp(min=0)
                z = float(w.sum())
        if not bool((w > 0).any()):
            w = probs[i, path[-1]].double()
        mass = torch.cumsum(w, 0)
        token = int((mass <= float(uniform[i, 0].double()) * float(mass[-1])).sum()) if float(mass[-1]) > 0 else -1
        found.append((len(path), path, token))
    return found
